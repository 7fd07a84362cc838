// Stand-in for the HIP runtime under the objects of the row operators: a launch
// is recorded, nothing runs, and one that the runtime would refuse is refused.
// Kernels with a map of rows to workgroups are recorded with it, the others with
// the row of their first workgroup.
#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <iterator>
#include <map>
#include <string>
#include <vector>

#include "rows_internal.h"

namespace {

struct Launch {
  std::string name;
  uint64_t blocks, threads;
  int first, parts, bits;
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

bool has(const std::string& s, const char* part) { return s.find(part) != std::string::npos; }

}  // namespace

namespace qmoe {   // of the layer's boundary, which is not linked here
moe_status hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }
bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
}  // namespace qmoe

extern "C" {

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
  Launch l{names()[f], grid.x, block.x, 0, 0, -1};
  if (has(l.name, "RowMap")) {
    const qmoe::RowMap& m = *static_cast<const qmoe::RowMap*>(args[1]);
    l.first = m.first;
    l.parts = m.parts;
    l.bits = m.bits;
  } else if (has(l.name, "swiglu_e4m3")) {
    l.first = static_cast<const qmoe::SwigluArgs*>(args[0])->first;
  } else if (has(l.name, "8NormArgs")) {
    l.first = static_cast<const qmoe::NormArgs*>(args[0])->first;
  } else if (has(l.name, "collect_grad")) {
    l.parts = *static_cast<const int*>(args[1]);   // picks a workgroup
  }
  launches.push_back(l);
  const bool fits = grid.x > 0 && l.blocks * l.threads < (1ull << 32) && grid.y == 1 && grid.z == 1 && block.x <= 1024;
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
int recorded_parts(int i) { return launches[i].parts; }
int recorded_bits(int i) { return launches[i].bits; }

}  // extern "C"
