// Stand-in for the HIP runtime under the objects of the MXFP4 and
// router-balance operators: a launch is recorded, nothing runs.  So a test
// without a GPU sees which kernels a call takes and the shape of each launch,
// and a launch that the runtime would refuse (2^32 work items and more along x)
// is refused here too.
#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <cstring>
#include <iterator>
#include <map>
#include <string>
#include <vector>

#include "operators_internal.h"

namespace {

struct Launch {
  std::string name;   // as the compiler mangles it
  uint64_t blocks, threads;
  qmoe::MxQuantArgs quant;   // of a conversion
  int first;                 // of a few-row product: its first unit of rows
};
struct Shape {
  dim3 grid, block;
  size_t lds;
  hipStream_t stream;
};

std::map<const void*, std::string>& names() {
  static std::map<const void*, std::string> m;
  return m;
}
std::vector<Launch> launches;
std::vector<Shape> shapes;
hipError_t last = hipSuccess;

}  // namespace

namespace qmoe {   // of the layer's boundary, which is not linked here
moe_status hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }
bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
}  // namespace qmoe

extern "C" {

// what the objects' own start-up and launch stubs call
int __hip_fatbin_token;
void** __hipRegisterFatBinary(const void*) { return reinterpret_cast<void**>(&__hip_fatbin_token); }
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* host, char*, const char* device, unsigned, void*, void*, void*, void*, int*) {
  names()[host] = device;
}
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, hipStream_t stream) {
  shapes.push_back({grid, block, lds, stream});
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, hipStream_t* stream) {
  const Shape s = shapes.back();
  shapes.pop_back();
  *grid = s.grid;
  *block = s.block;
  *lds = s.lds;
  *stream = s.stream;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void* f, dim3 grid, dim3 block, void** args, size_t, hipStream_t) {
  Launch l{};
  l.name = names()[f];
  l.blocks = grid.x;
  l.threads = (uint64_t)grid.x * block.x;
  if (l.name.find("quantize_kernel") != std::string::npos) std::memcpy(&l.quant, args[0], sizeof l.quant);
  if (l.name.find("mx_matmul_thin") != std::string::npos) l.first = *static_cast<int*>(args[3]);
  if (l.name.find("mx_matmul_dx_thin") != std::string::npos) l.first = *static_cast<int*>(args[2]);
  launches.push_back(l);
  const bool fits = grid.x > 0 && l.threads < (1ull << 32) && grid.y == 1 && grid.z == 1 && block.x <= 1024;
  return last = fits ? hipSuccess : hipErrorInvalidConfiguration;
}
hipError_t hipGetLastError() {
  const hipError_t e = last;
  last = hipSuccess;
  return e;
}

int registered() { return (int)names().size(); }
const char* registered_name(int i) { return std::next(names().begin(), i)->second.c_str(); }
int recorded() { return (int)launches.size(); }
void forget() { launches.clear(); }
const char* recorded_name(int i) { return launches[i].name.c_str(); }
uint64_t recorded_blocks(int i) { return launches[i].blocks; }
uint64_t recorded_threads(int i) { return launches[i].threads; }
int recorded_first(int i) { return launches[i].first; }
int64_t recorded_rows(int i) { return launches[i].quant.rows; }
uint64_t recorded_x(int i) { return (uint64_t) reinterpret_cast<uintptr_t>(launches[i].quant.x); }
uint64_t recorded_codes(int i) { return (uint64_t) reinterpret_cast<uintptr_t>(launches[i].quant.codes); }
uint64_t recorded_scale(int i) { return (uint64_t) reinterpret_cast<uintptr_t>(launches[i].quant.scale); }

}  // extern "C"
