// Stand-ins for the HIP runtime calls that the library's host code makes: a
// launch is written down (kernel, grid, first argument) and nothing runs, so
// that which kernel a call launches, on what, can be checked without a GPU.
#include <cstdint>
#include <cstring>
#include <map>
#include <string>
#include <vector>

namespace {

struct Dim3 {
    uint32_t x, y, z;
};
struct Launch {
    const char* name;
    Dim3 grid, block;
    size_t lds;
    const void* args;                  // the first argument, copied
    size_t bytes;
};

std::map<const void*, std::string>& names() {
    static std::map<const void*, std::string> m;
    return m;
}
std::vector<std::pair<Launch, std::vector<uint8_t>>> g_launches;
Dim3 g_grid, g_block;
size_t g_lds;
void* g_stream;
size_t g_arg_bytes = 0;                // how much of the first argument to keep

int record(const void* f, Dim3 grid, Dim3 block, void** args, size_t lds) {
    const auto it = names().find(f);
    const uint8_t* const a = static_cast<const uint8_t*>(args[0]);
    g_launches.push_back({{it == names().end() ? "" : it->second.c_str(), grid, block, lds, nullptr, 0},
                          std::vector<uint8_t>(a, a + g_arg_bytes)});
    return 0;
}

}  // namespace

extern "C" {

void** __hipRegisterFatBinary(const void*) {
    static void* handle;
    return &handle;
}
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* f, char*, const char* name, unsigned, void*, void*, void*, void*, int*) {
    names()[f] = name;
}
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
int __hipPushCallConfiguration(Dim3 grid, Dim3 block, size_t lds, void* stream) {
    g_grid = grid;
    g_block = block;
    g_lds = lds;
    g_stream = stream;
    return 0;
}
int __hipPopCallConfiguration(Dim3* grid, Dim3* block, size_t* lds, void** stream) {
    *grid = g_grid;
    *block = g_block;
    *lds = g_lds;
    *stream = g_stream;
    return 0;
}
int hipLaunchKernel(const void* f, Dim3 grid, Dim3 block, void** args, size_t lds, void*) {
    return record(f, grid, block, args, lds);
}
int hipExtLaunchKernel(const void* f, Dim3 grid, Dim3 block, void** args, size_t lds, void*, void*, void*, int) {
    return record(f, grid, block, args, lds);
}
int hipGetLastError() { return 0; }
const char* hipGetErrorString(int) { return "error"; }
int hipGetDevice(int* d) {
    *d = 0;
    return 0;
}
int hipDeviceGetAttribute(int* v, int, int) {
    *v = 256;                          // compute units
    return 0;
}

// What the tests read.
int recorded_kernels() { return int(names().size()); }
const char* recorded_kernel(int i) {
    auto it = names().begin();
    while (i-- > 0) ++it;
    return it->second.c_str();
}
void record_start(uint64_t arg_bytes) {
    g_launches.clear();
    g_arg_bytes = arg_bytes;
}
int recorded_launches() { return int(g_launches.size()); }
const char* recorded_launch(int i, uint32_t dims[6], uint64_t* lds, uint8_t* args) {
    const auto& l = g_launches[size_t(i)];
    const Dim3 g = l.first.grid, b = l.first.block;
    const uint32_t d[6] = {g.x, g.y, g.z, b.x, b.y, b.z};
    std::memcpy(dims, d, sizeof d);
    *lds = l.first.lds;
    if (args && !l.second.empty()) std::memcpy(args, l.second.data(), l.second.size());
    return l.first.name;
}

}  // extern "C"
