/*
 * The experts' entry points linked against a stand-in for the CUDA runtime, so that what they do on the host can be
 * seen without a GPU: the stand-in reports a device of the compute capability given as the first argument, counts
 * launches, keeps the grid of the last one and runs nothing.  Prints a line for each call: name, status, launches,
 * grid.  No pointer is dereferenced.
 */
#include <stdio.h>
#include <stdlib.h>

#include "moe_route.h"

typedef struct {
    unsigned x, y, z;
} Dim3;

static int g_major, g_launches;
static Dim3 g_grid;

/* ---- the runtime that the library's objects call */
int cudaGetDevice(int *dev)
{
    *dev = 0;
    return 0;
}
int cudaDeviceGetAttribute(int *v, int attr, int dev)
{
    (void)dev;
    *v = attr == 75 ? g_major : attr == 16 ? 152 : 1 << 20; /* capability, multiprocessors, anything else */
    return 0;
}
int cudaFuncSetAttribute(const void *f, int attr, int value)
{
    (void)f, (void)attr, (void)value;
    return 0;
}
static int encode(void) { return 0; }
int cudaGetDriverEntryPointByVersion(const char *name, void **fn, unsigned version, unsigned long long flags, int *result)
{
    (void)name, (void)version, (void)flags;
    *fn = (void *)encode;
    *result = 0;
    return 0;
}
int cudaGetLastError(void) { return 0; }
static int launched(Dim3 grid)
{
    ++g_launches;
    g_grid = grid;
    return 0;
}
int cudaLaunchKernelExC(const Dim3 *cfg, const void *f, void **args)
{
    (void)f, (void)args;
    return launched(*cfg); /* the grid is a launch configuration's first member */
}
int __cudaPushCallConfiguration(Dim3 grid, Dim3 block, size_t shared, void *stream)
{
    (void)block, (void)shared, (void)stream;
    g_grid = grid;
    return 0;
}
int __cudaPopCallConfiguration(Dim3 *grid, Dim3 *block, size_t *shared, void *stream)
{
    Dim3 one = {1, 1, 1};
    *grid = g_grid;
    *block = one;
    *shared = 0;
    *(void **)stream = NULL;
    return 0;
}
int __cudaGetKernel(void **kernel, const void *f)
{
    *kernel = (void *)f;
    return 0;
}
int __cudaLaunchKernel(void *kernel, Dim3 grid, Dim3 block, void **args, size_t shared, void *stream)
{
    (void)kernel, (void)block, (void)args, (void)shared, (void)stream;
    return launched(grid);
}
void **__cudaRegisterFatBinary(void *image)
{
    static void *handle;
    (void)image;
    return &handle;
}
void __cudaRegisterFatBinaryEnd(void **handle) { (void)handle; }
void __cudaUnregisterFatBinary(void **handle) { (void)handle; }
void __cudaRegisterFunction(void) {}
void __cudaRegisterVar(void) {}
int cudaGetSymbolAddress(void **p, const void *symbol)
{
    *p = (void *)symbol;
    return 0;
}
int cudaMemsetAsync(void) { return 0; }
int cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int *n)
{
    return *n = 1, 0;
}
int cudaOccupancyMaxActiveClusters(int *n)
{
    return *n = 1, 0;
}

/* ---- the calls */
static void report(const char *name, int status)
{
    printf("%s %d %d %u %u %u\n", name, status, g_launches, g_grid.x, g_grid.y, g_grid.z);
    g_launches = 0;
}

int main(int argc, char **argv)
{
    char *a = (char *)0x10000, *b = (char *)0x20000, *c = (char *)0x30000, *d = (char *)0x40000, *e = (char *)0x50000;
    g_major = argc > 1 ? atoi(argv[1]) : 10;
    report("moe_quantize_weight", moe_quantize_weight(a, 2, 256, 256, b, c, 0, NULL));
    report("moe_expert_gemm", moe_expert_gemm(a, b, 0, c, d, 0, (int32_t *)e, 64, 4, 256, 128, 0, a, NULL, NULL));
    report("moe_expert_wgrad", moe_expert_wgrad(a, b, c, 0, (int32_t *)d, 64, 4, 256, 128, NULL, e, 0, NULL, NULL));
    report("moe_swiglu", moe_swiglu(a, 64, 128, b, c, d, e, 0, NULL));
    report("moe_swiglu_backward", moe_swiglu_backward(a, b, c, 0, 64, 128, d, NULL, NULL, 0, NULL, NULL));
    report("moe_layer", moe_layer(a, b, NULL, c, d, e, a, 0, NULL, 4, 256, 128, 8, 2, 1, (int32_t *)b, (float *)c, d, NULL,
                                  a, moe_layer_workspace_size(4, 256, 128, 8, 2), NULL));
    /* the widest row that an int counts in whole eights */
    report("moe_quantize_weight:widest", moe_quantize_weight(a, 1, 1, 2147483640, b, c, 0, NULL));
    return 0;
}
