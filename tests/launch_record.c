/* A stand-in for the CUDA runtime under the library's host code: launches go into a list instead of to a device, and what the
 * device says of itself is set by the test. */
#include <cuda_runtime_api.h>
#include <stdlib.h>
#include <string.h>

typedef struct {
    const char* name;       /* mangled */
    unsigned grid[3], block[3], cluster;
    int smem, allowed, portable;
} record_t;

enum { kMost = 4096 };
static struct { const void* host; const char* name; int allowed, lowered, nonportable; } kernels[kMost];
static int n_kernels;
static record_t records[kMost];
static int n_records;
static int sms = 152, largest_cluster = 16;
static char symbol[256];

static int index_of(const void* host) {
    for (int i = 0; i < n_kernels; ++i)
        if (kernels[i].host == host) return i;
    abort();
}

void fake_device(int sm_count, int cluster) { sms = sm_count; largest_cluster = cluster; }
int fake_records(const record_t** at) { *at = records; return n_records; }
void fake_clear(void) { n_records = 0; }
/* kernels whose limit of dynamic shared memory was once taken below an earlier one */
int fake_lowered(void) {
    int n = 0;
    for (int i = 0; i < n_kernels; ++i) n += kernels[i].lowered;
    return n;
}

/* what nvcc's objects register and call */
void** __cudaRegisterFatBinary(void* x) { return (void**)x; }
void __cudaRegisterFatBinaryEnd(void** h) { (void)h; }
void __cudaUnregisterFatBinary(void** h) { (void)h; }
void __cudaRegisterVar(void** h, char* host, char* dev, const char* name, int ext, size_t size, int constant, int global) {
    (void)h; (void)host; (void)dev; (void)name; (void)ext; (void)size; (void)constant; (void)global;
}
void __cudaRegisterFunction(void** h, const char* host, char* dev, const char* name, int limit, void* tid, void* bid, void* bdim, void* gdim, int* wsize) {
    (void)h; (void)dev; (void)limit; (void)tid; (void)bid; (void)bdim; (void)gdim; (void)wsize;
    if (n_kernels == kMost) abort();
    kernels[n_kernels].host = host;
    kernels[n_kernels].name = name;
    kernels[n_kernels++].allowed = 48 * 1024;
}
cudaError_t __cudaGetKernel(void** k, const void* f) { *k = (void*)f; return cudaSuccess; }
unsigned __cudaPushCallConfiguration(dim3 g, dim3 b, size_t s, void* st) { (void)g; (void)b; (void)s; (void)st; return 1; }
cudaError_t __cudaPopCallConfiguration(dim3* g, dim3* b, size_t* s, void* st) { (void)g; (void)b; (void)s; (void)st; return cudaErrorUnknown; }
cudaError_t __cudaLaunchKernel(void* k, dim3 g, dim3 b, void** a, size_t s, void* st) {
    (void)k; (void)g; (void)b; (void)a; (void)s; (void)st;
    return cudaErrorUnknown;
}

cudaError_t cudaFuncSetAttribute(const void* f, enum cudaFuncAttribute what, int value) {
    const int i = index_of(f);
    if (what == cudaFuncAttributeMaxDynamicSharedMemorySize) {
        if (value > 227 * 1024) return cudaErrorInvalidValue;
        if (value < kernels[i].allowed && kernels[i].allowed != 48 * 1024) kernels[i].lowered = 1;
        kernels[i].allowed = value;
    }
    if (what == cudaFuncAttributeNonPortableClusterSizeAllowed) kernels[i].nonportable = value;
    return cudaSuccess;
}
static unsigned cluster_of(const cudaLaunchConfig_t* c) {
    for (unsigned i = 0; i < c->numAttrs; ++i)
        if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) return c->attrs[i].val.clusterDim.x;
    return 1;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void** args) {
    (void)args;
    const int i = index_of(f);
    const unsigned cluster = cluster_of(c);
    if ((int)c->dynamicSmemBytes > kernels[i].allowed) return cudaErrorInvalidValue;
    if ((int)cluster > largest_cluster || (cluster > 8 && !kernels[i].nonportable) || c->gridDim.x % cluster != 0) return cudaErrorInvalidClusterSize;
    if (n_records == kMost) abort();
    record_t r = {kernels[i].name, {c->gridDim.x, c->gridDim.y, c->gridDim.z}, {c->blockDim.x, c->blockDim.y, c->blockDim.z}, cluster,
                  (int)c->dynamicSmemBytes, kernels[i].allowed, !kernels[i].nonportable};
    records[n_records++] = r;
    return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void* f, const cudaLaunchConfig_t* c) {
    const int i = index_of(f);
    const int size = (int)cluster_of(c);
    if (size > 8 && !kernels[i].nonportable) return cudaErrorInvalidClusterSize;
    *n = size <= largest_cluster ? sms / size : 0;
    return cudaSuccess;
}
cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, enum cudaDeviceAttr a, int d) {
    (void)d;
    *v = a == cudaDevAttrMultiProcessorCount ? sms : 0;
    return cudaSuccess;
}
cudaError_t cudaGetSymbolAddress(void** p, const void* s) { (void)s; *p = symbol; return cudaSuccess; }
const char* cudaGetErrorName(cudaError_t e) { return e == cudaErrorInvalidClusterSize ? "cluster size" : e == cudaSuccess ? "none" : "error"; }
const char* cudaGetErrorString(cudaError_t e) { return cudaGetErrorName(e); }
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
cudaError_t cudaDeviceSynchronize(void) { return cudaSuccess; }

/* not reached by the calls that are recorded */
cudaError_t cudaEventCreateWithFlags(cudaEvent_t* e, unsigned f) { (void)e; (void)f; return cudaErrorUnknown; }
cudaError_t cudaEventRecord(cudaEvent_t e, cudaStream_t s) { (void)e; (void)s; return cudaErrorUnknown; }
cudaError_t cudaStreamCreateWithFlags(cudaStream_t* s, unsigned f) { (void)s; (void)f; return cudaErrorUnknown; }
cudaError_t cudaStreamWaitEvent(cudaStream_t s, cudaEvent_t e, unsigned f) { (void)s; (void)e; (void)f; return cudaErrorUnknown; }
cudaError_t cudaGetDriverEntryPointByVersion(const char* n, void** p, unsigned v, unsigned long long f, enum cudaDriverEntryPointQueryResult* r) {
    (void)n; (void)p; (void)v; (void)f; (void)r;
    return cudaErrorUnknown;
}
cudaError_t cudaMemcpyAsync(void* d, const void* s, size_t n, enum cudaMemcpyKind k, cudaStream_t t) {
    (void)d; (void)s; (void)n; (void)k; (void)t;
    return cudaErrorUnknown;
}
cudaError_t cudaMemcpy2DAsync(void* d, size_t dp, const void* s, size_t sp, size_t w, size_t h, enum cudaMemcpyKind k, cudaStream_t t) {
    (void)d; (void)dp; (void)s; (void)sp; (void)w; (void)h; (void)k; (void)t;
    return cudaErrorUnknown;
}
cudaError_t cudaMemcpyFromSymbol(void* d, const void* s, size_t n, size_t o, enum cudaMemcpyKind k) {
    (void)d; (void)s; (void)n; (void)o; (void)k;
    return cudaErrorUnknown;
}
cudaError_t cudaMemcpyToSymbol(const void* d, const void* s, size_t n, size_t o, enum cudaMemcpyKind k) {
    (void)d; (void)s; (void)n; (void)o; (void)k;
    return cudaErrorUnknown;
}
