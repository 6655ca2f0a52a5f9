// A CUDA runtime without a GPU, for tests of what the library does on the host: which kernels a call launches, in what
// order and how, and what it leaves behind when a runtime call fails.  Launches are written to a log; those of a
// capturing stream go into a graph and to the log when the graph is launched.  Linked with the library's objects in place
// of the CUDA runtime.
#include <cuda.h>
#include <cuda_runtime_api.h>
#include <cxxabi.h>
#include <stdlib.h>
#include <string.h>

#include <map>
#include <string>
#include <vector>

namespace {

struct Graph {
    std::vector<std::string> launches;
};
struct Config {
    dim3 grid, block;
    size_t smem;
    cudaStream_t stream;
};

std::map<const void*, std::string>& names() {
    static std::map<const void*, std::string> m;
    return m;
}
std::map<cudaStream_t, Graph*> capturing;
std::map<std::string, std::pair<int, int>> failing;   // function: calls until it fails, error
std::vector<Config> configs;
std::string log_text;
cudaError_t last = cudaSuccess;
cudaGraphNode_t last_node = nullptr;
long handles = 0x1000;

cudaError_t done(const char* fn) {
    auto it = failing.find(fn);
    if (it == failing.end() || --it->second.first != 0) return cudaSuccess;
    return last = (cudaError_t)it->second.second;
}
#define CALL(fn)                          \
    do {                                  \
        const cudaError_t e_ = done(#fn); \
        if (e_ != cudaSuccess) return e_; \
    } while (0)

void record(cudaStream_t s, const std::string& line) {
    auto it = capturing.find(s);
    if (it == capturing.end()) {
        log_text += line + "\n";
        return;
    }
    it->second->launches.push_back(line);
    last_node = (cudaGraphNode_t)(it->second->launches.size());
}

std::string kernel(const void* f) {
    auto it = names().find(f);
    if (it == names().end()) return "?";
    int st = 0;
    char* d = abi::__cxa_demangle(it->second.c_str(), nullptr, nullptr, &st);
    std::string s = st == 0 ? d : it->second;
    free(d);
    const size_t at = s.find("(");
    s = s.substr(0, at);
    const size_t colons = s.rfind("vc::", s.find('<'));
    return colons == std::string::npos ? s : s.substr(colons + 4);
}

CUresult encode_tiled(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                      const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                      CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
    return CUDA_SUCCESS;
}

}  // namespace

extern "C" {

// ---- the tests' side -----------------------------------------------------------------------------
const char* fake_log() { return log_text.c_str(); }
void fake_reset() {
    log_text.clear();
    failing.clear();
    last = cudaSuccess;
}
// the n-th call of fn from now on returns err
void fake_fail(const char* fn, int n, int err) { failing[fn] = {n, err}; }

// ---- launches ------------------------------------------------------------------------------------
void** __cudaRegisterFatBinary(void*) {
    static void* h = nullptr;
    return &h;
}
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char* host, char*, const char* name, int, uint3*, uint3*, dim3*, dim3*, int*) {
    names()[host] = name;
}
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}
unsigned __cudaPushCallConfiguration(dim3 grid, dim3 block, size_t smem, struct CUstream_st* stream) {
    configs.push_back({grid, block, smem, stream});
    return 0;
}
cudaError_t __cudaPopCallConfiguration(dim3* grid, dim3* block, size_t* smem, void* stream) {
    const Config c = configs.back();
    configs.pop_back();
    *grid = c.grid;
    *block = c.block;
    *smem = c.smem;
    *(cudaStream_t*)stream = c.stream;
    return cudaSuccess;
}
cudaError_t cudaLaunchKernel(const void* f, dim3, dim3, void**, size_t, cudaStream_t s) {
    CALL(cudaLaunchKernel);
    record(s, kernel(f));
    return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
    CALL(cudaLaunchKernelExC);
    bool pdl = false;
    for (unsigned i = 0; i < c->numAttrs; ++i)
        pdl |= c->attrs[i].id == cudaLaunchAttributeProgrammaticStreamSerialization &&
               c->attrs[i].val.programmaticStreamSerializationAllowed;
    record(c->stream, kernel(f) + (pdl ? " pdl" : ""));
    return cudaSuccess;
}
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t s) {
    CALL(cudaMemsetAsync);
    record(s, "memset");
    return cudaSuccess;
}
cudaError_t cudaMemcpyAsync(void*, const void*, size_t, cudaMemcpyKind, cudaStream_t s) {
    CALL(cudaMemcpyAsync);
    record(s, "memcpy");
    return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return done("cudaFuncSetAttribute"); }
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int* n, const void*, int, size_t, unsigned) {
    *n = 1;
    return cudaSuccess;
}

// ---- graphs --------------------------------------------------------------------------------------
cudaError_t cudaStreamBeginCapture(cudaStream_t s, cudaStreamCaptureMode) {
    CALL(cudaStreamBeginCapture);
    capturing[s] = new Graph;
    return cudaSuccess;
}
cudaError_t cudaStreamEndCapture(cudaStream_t s, cudaGraph_t* g) {
    Graph* graph = capturing[s];
    capturing.erase(s);
    *g = nullptr;
    CALL(cudaStreamEndCapture);
    *g = (cudaGraph_t)graph;
    return cudaSuccess;
}
cudaError_t cudaStreamGetCaptureInfo_v2(cudaStream_t s, cudaStreamCaptureStatus* st, unsigned long long*, cudaGraph_t* g,
                                        const cudaGraphNode_t** deps, size_t* n) {
    CALL(cudaStreamGetCaptureInfo);
    auto it = capturing.find(s);
    *st = it == capturing.end() ? cudaStreamCaptureStatusNone : cudaStreamCaptureStatusActive;
    if (it == capturing.end()) return cudaSuccess;
    if (g) *g = (cudaGraph_t)it->second;
    if (deps) *deps = &last_node;
    if (n) *n = 1;
    return cudaSuccess;
}
cudaError_t cudaGraphGetRootNodes(cudaGraph_t, cudaGraphNode_t* nodes, size_t* n) {
    if (nodes) nodes[0] = (cudaGraphNode_t)1;
    *n = 1;
    return cudaSuccess;
}
cudaError_t cudaGraphInstantiate(cudaGraphExec_t* e, cudaGraph_t g, unsigned long long) {
    CALL(cudaGraphInstantiate);
    *e = (cudaGraphExec_t)g;
    return cudaSuccess;
}
cudaError_t cudaGraphLaunch(cudaGraphExec_t e, cudaStream_t) {
    CALL(cudaGraphLaunch);
    for (const std::string& l : ((Graph*)e)->launches) log_text += l + "\n";
    return cudaSuccess;
}
cudaError_t cudaGraphKernelNodeGetParams(cudaGraphNode_t, cudaKernelNodeParams*) { return cudaErrorNotSupported; }
cudaError_t cudaGraphExecKernelNodeSetParams(cudaGraphExec_t, cudaGraphNode_t, const cudaKernelNodeParams*) {
    return cudaErrorNotSupported;
}
cudaError_t cudaGraphExecDestroy(cudaGraphExec_t) { return cudaSuccess; }
cudaError_t cudaGraphDestroy(cudaGraph_t g) {
    delete (Graph*)g;
    return cudaSuccess;
}

// ---- the rest ------------------------------------------------------------------------------------
cudaError_t cudaStreamCreateWithFlags(cudaStream_t* s, unsigned) {
    *s = (cudaStream_t)(handles += 16);
    return done("cudaStreamCreateWithFlags");
}
cudaError_t cudaStreamDestroy(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamWaitEvent(cudaStream_t, cudaEvent_t, unsigned) { return done("cudaStreamWaitEvent"); }
cudaError_t cudaEventCreateWithFlags(cudaEvent_t* e, unsigned) {
    *e = (cudaEvent_t)(handles += 16);
    return done("cudaEventCreateWithFlags");
}
cudaError_t cudaEventDestroy(cudaEvent_t) { return cudaSuccess; }
cudaError_t cudaEventRecord(cudaEvent_t, cudaStream_t) { return done("cudaEventRecord"); }
cudaError_t cudaGetDevice(int* d) {
    *d = 0;
    return done("cudaGetDevice");
}
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int) {
    *v = a == cudaDevAttrMultiProcessorCount ? 148 : 0;
    return done("cudaDeviceGetAttribute");
}
cudaError_t cudaGetLastError() {
    const cudaError_t e = last;
    last = cudaSuccess;
    return e;
}
const char* cudaGetErrorString(cudaError_t) { return "an error of the fake runtime"; }
cudaError_t cudaGetSymbolAddress(void** p, const void* s) {
    *p = (void*)s;
    return cudaSuccess;
}
cudaError_t cudaGetDriverEntryPoint(const char*, void** f, unsigned long long, cudaDriverEntryPointQueryResult* r) {
    *f = (void*)&encode_tiled;
    if (r) *r = cudaDriverEntryPointSuccess;
    return done("cudaGetDriverEntryPoint");
}

}  // extern "C"
