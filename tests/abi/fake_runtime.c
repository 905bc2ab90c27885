/* A CUDA runtime of several devices that launches nothing: the library's host code runs against it without a GPU.
 * It keeps, as the real one does, the shared memory that each kernel was allowed on each device, and refuses launches
 * above it. Controls for the tests begin with fake_. Other runtime functions are generated by the test and fail. */
#include <cuda.h>
#include <cuda_runtime_api.h>
#include <stdlib.h>
#include <string.h>

#define KERNELS 256
#define DEVICES 4

static int device, fail_allowances, allowances, launches, encodes, pool_allocations;
static cudaLaunchConfig_t last;
static const void* kernels[KERNELS];
static int allowed[KERNELS][DEVICES];

static int kernel_index(const void* f) {
    int i = 0;
    while (i < KERNELS - 1 && kernels[i] && kernels[i] != f) ++i;
    kernels[i] = f;
    return i;
}

void fake_set_device(int d) { device = d; }
void fake_fail_allowances(int n) { fail_allowances = n; }
int fake_allowances(void) { return allowances; }
int fake_launches(void) { return launches; }
int fake_encodes(void) { return encodes; }
int fake_pool_allocations(void) { return pool_allocations; }
unsigned fake_last_grid(void) { return last.gridDim.x; }

cudaError_t cudaGetDevice(int* d) {
    *d = device;
    return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* v, enum cudaDeviceAttr a, int d) {
    *v = a == cudaDevAttrMultiProcessorCount ? (d == 0 ? 152 : 76) : 0;  /* the devices differ */
    return cudaSuccess;
}
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void* f, enum cudaFuncAttribute a, int v) {
    if (a != cudaFuncAttributeMaxDynamicSharedMemorySize) return cudaSuccess;
    ++allowances;
    if (fail_allowances > 0) {
        --fail_allowances;
        return cudaErrorMemoryAllocation;
    }
    allowed[kernel_index(f)][device] = v;
    return cudaSuccess;
}
static cudaError_t launch(const void* f, size_t smem) {
    const int most = allowed[kernel_index(f)][device];
    if (smem > (size_t)(most > 49152 ? most : 49152)) return cudaErrorInvalidValue;
    ++launches;
    return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void** args) {
    (void)args;
    last = *c;
    if (c->gridDim.x == 0 || c->gridDim.x > 0x7fffffffu) return cudaErrorInvalidConfiguration;
    return launch(f, c->dynamicSmemBytes);
}

/* launches in the <<< >>> form */
static size_t pushed_smem;
unsigned __cudaPushCallConfiguration(dim3 grid, dim3 block, size_t smem, struct CUstream_st* s) {
    (void)grid, (void)block, (void)s;
    pushed_smem = smem;
    return 0;
}
cudaError_t __cudaPopCallConfiguration(dim3* grid, dim3* block, size_t* smem, void* s) {
    memset(grid, 0, sizeof *grid);
    memset(block, 0, sizeof *block);
    *smem = pushed_smem;
    *(void**)s = 0;
    return cudaSuccess;
}
cudaError_t __cudaGetKernel(cudaKernel_t* k, const void* f) {
    *k = (cudaKernel_t)f;
    return cudaSuccess;
}
cudaError_t __cudaLaunchKernel(cudaKernel_t k, dim3 grid, dim3 block, void** args, size_t smem, cudaStream_t s) {
    (void)grid, (void)block, (void)args, (void)s;
    return launch((const void*)k, smem);
}

/* what the object files do when they are loaded */
void** __cudaRegisterFatBinary(void* b) {
    (void)b;
    return calloc(1, sizeof(void*));
}
void __cudaRegisterFatBinaryEnd(void** h) { (void)h; }
void __cudaUnregisterFatBinary(void** h) { free(h); }
void __cudaRegisterFunction(void** h, const char* f, char* n, const char* d, int t, void* a, void* b, void* c, void* e, int* w) {
    (void)h, (void)f, (void)n, (void)d, (void)t, (void)a, (void)b, (void)c, (void)e, (void)w;
}
void __cudaRegisterVar(void** h, char* v, char* a, const char* n, int e, size_t s, int c, int g) {
    (void)h, (void)v, (void)a, (void)n, (void)e, (void)s, (void)c, (void)g;
}

/* memory: host words are real, device addresses only have to be aligned */
cudaError_t cudaHostAlloc(void** p, size_t n, unsigned flags) {
    (void)flags;
    return (*p = calloc(1, n)) ? cudaSuccess : cudaErrorMemoryAllocation;
}
cudaError_t cudaHostGetDevicePointer(void** d, void* h, unsigned flags) {
    (void)flags;
    *d = h;
    return cudaSuccess;
}
cudaError_t cudaMemPoolCreate(cudaMemPool_t* p, const struct cudaMemPoolProps* props) {
    *p = (cudaMemPool_t)(size_t)(0x100 + props->location.id);
    return cudaSuccess;
}
cudaError_t cudaMemPoolSetAttribute(cudaMemPool_t p, enum cudaMemPoolAttr a, void* v) {
    (void)p, (void)a, (void)v;
    return cudaSuccess;
}
cudaError_t cudaMallocFromPoolAsync(void** p, size_t n, cudaMemPool_t pool, cudaStream_t s) {
    (void)n, (void)pool, (void)s;
    ++pool_allocations;
    *p = (void*)((size_t)1 << 40);
    return cudaSuccess;
}
cudaError_t cudaFreeAsync(void* p, cudaStream_t s) {
    (void)p, (void)s;
    return cudaSuccess;
}

static CUresult encode(CUtensorMap* m, CUtensorMapDataType t, cuuint32_t rank, void* p, const cuuint64_t* dims,
                       const cuuint64_t* strides, const cuuint32_t* box, const cuuint32_t* elem, CUtensorMapInterleave i,
                       CUtensorMapSwizzle s, CUtensorMapL2promotion l, CUtensorMapFloatOOBfill f) {
    (void)m, (void)t, (void)rank, (void)p, (void)dims, (void)strides, (void)box, (void)elem, (void)i, (void)s, (void)l, (void)f;
    ++encodes;
    return CUDA_SUCCESS;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char* name, void** f, unsigned version, unsigned long long flags,
                                             enum cudaDriverEntryPointQueryResult* q) {
    (void)version, (void)flags;
    *f = strcmp(name, "cuTensorMapEncodeTiled") ? 0 : (void*)encode;
    *q = *f ? cudaDriverEntryPointSuccess : cudaDriverEntryPointSymbolNotFound;
    return cudaSuccess;
}
