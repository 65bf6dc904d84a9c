// A stand-in for the CUDA runtime, for tests of the library's host code on a
// machine without a GPU: launches are noted and return, device variables live in
// their host shadows, and launches, occupancy queries and allocations can be made
// to fail.
#include <cstdlib>
#include <cstring>
#include <new>
#include <string>
#include <vector>

#include <cuda_runtime_api.h>

namespace {

struct Launch {
    std::string name;
    unsigned grid;
    const void *arg0;
    int arg1;
};

std::vector<std::pair<const void *, std::string>> functions, variables;
std::vector<Launch> launches;
int fail_at = -1, fail_queries = 0, fail_call = 0;
bool no_memory = false;
cudaError_t last = cudaSuccess;
void *handle = nullptr;

int encode_tiled() { return 0; }

struct Allow {  // the fake's own allocations
    bool was = no_memory;
    Allow() { no_memory = false; }
    ~Allow() { no_memory = was; }
};

bool fails() { return fail_call > 0 && --fail_call == 0; }

std::string name_of(const void *f)
{
    for (auto &p : functions)
        if (p.first == f)
            return p.second;
    return "?";
}

}  // namespace

void *operator new(std::size_t n)
{
    void *p = no_memory ? nullptr : std::malloc(n);
    if (p == nullptr)
        throw std::bad_alloc();
    return p;
}
void operator delete(void *p) noexcept { std::free(p); }
void operator delete(void *p, std::size_t) noexcept { std::free(p); }

extern "C" {

// ---- what the tests ask ---------------------------------------------------------
void fake_reset(int fail)  // the launch number `fail` fails (-1: none)
{
    launches.clear();
    fail_at = fail;
    fail_queries = fail_call = 0;
    no_memory = false;
    last = cudaSuccess;
}
void fake_fail_queries(int n) { fail_queries = n; }  // the next n occupancy queries fail
void fake_fail_call(int n) { fail_call = n; }         // the n-th call of the runtime from here on fails, launches not counted
int fake_calls_left() { return fail_call; }           // 0: it has failed
void fake_no_memory(int on) { no_memory = on != 0; }  // operator new throws in the library's code
int fake_launches() { return static_cast<int>(launches.size()); }
const char *fake_launch_name(int i) { return launches[i].name.c_str(); }
unsigned fake_launch_grid(int i) { return launches[i].grid; }
const void *fake_launch_arg0(int i) { return launches[i].arg0; }
int fake_launch_arg1(int i) { return launches[i].arg1; }
// the i-th device variable whose name holds `part`
void *fake_variable(const char *part, int i)
{
    for (auto &p : variables)
        if (p.second.find(part) != std::string::npos && i-- == 0)
            return const_cast<void *>(p.first);
    return nullptr;
}

// ---- the runtime ------------------------------------------------------------------
void **__cudaRegisterFatBinary(void *) { return &handle; }
void __cudaRegisterFatBinaryEnd(void **) {}
void __cudaUnregisterFatBinary(void **) {}
void __cudaRegisterFunction(void **, const char *host, char *, const char *name, int, uint3 *, uint3 *, dim3 *, dim3 *, int *)
{
    functions.emplace_back(host, name);
}
void __cudaRegisterVar(void **, char *host, char *, const char *name, int, size_t, int, int)
{
    variables.emplace_back(host, name);
}
unsigned __cudaPopCallConfiguration(dim3 *, dim3 *, size_t *, void *) { return cudaErrorInvalidConfiguration; }

cudaError_t cudaGetDevice(int *d)
{
    if (fails())
        return last = cudaErrorInvalidValue;
    *d = 0;
    return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr a, int)
{
    if (fails())
        return last = cudaErrorInvalidValue;
    *v = a == cudaDevAttrMultiProcessorCount ? 148 : 0;
    return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int)
{
    return fails() ? last = cudaErrorInvalidValue : cudaSuccess;
}
cudaError_t cudaGetDriverEntryPoint(const char *, void **f, unsigned long long, cudaDriverEntryPointQueryResult *r)
{
    if (fails())
        return last = cudaErrorInvalidValue;
    *f = reinterpret_cast<void *>(&encode_tiled);
    *r = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}
cudaError_t cudaGetLastError()
{
    const cudaError_t e = last;
    last = cudaSuccess;
    return e;
}
cudaError_t cudaPeekAtLastError() { return last; }
cudaError_t cudaGetSymbolAddress(void **p, const void *symbol)
{
    if (fails())
        return last = cudaErrorInvalidValue;
    *p = const_cast<void *>(symbol);
    return cudaSuccess;
}
cudaError_t cudaLaunchKernel(const void *, dim3, dim3, void **, size_t, cudaStream_t) { return last = cudaErrorLaunchFailure; }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *f, void **args)
{
    Allow a;
    Launch l{name_of(f), c->gridDim.x, nullptr, 0};
    if (l.name.find("clear") != std::string::npos) {  // (int *, int)
        std::memcpy(&l.arg0, args[0], sizeof l.arg0);
        std::memcpy(&l.arg1, args[1], sizeof l.arg1);
    }
    launches.push_back(l);
    if (fake_launches() - 1 == fail_at)
        return last = cudaErrorLaunchOutOfResources;
    return cudaSuccess;
}
cudaError_t cudaMemcpyFromSymbol(void *dst, const void *symbol, size_t n, size_t offset, cudaMemcpyKind)
{
    std::memcpy(dst, static_cast<const char *>(symbol) + offset, n);
    return cudaSuccess;
}
cudaError_t cudaMemcpyToSymbol(const void *symbol, const void *src, size_t n, size_t offset, cudaMemcpyKind)
{
    std::memcpy(static_cast<char *>(const_cast<void *>(symbol)) + offset, src, n);
    return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int *n, const void *, int, size_t, unsigned)
{
    if (fails())
        return last = cudaErrorInvalidValue;
    if (fail_queries > 0 && fail_queries-- > 0)
        return last = cudaErrorInvalidValue;
    *n = 1;
    return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int *n, const void *, const cudaLaunchConfig_t *)
{
    if (fails())
        return last = cudaErrorInvalidValue;
    if (fail_queries > 0 && fail_queries-- > 0)
        return last = cudaErrorInvalidValue;
    *n = 148 / 2;
    return cudaSuccess;
}
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }

}  // extern "C"
