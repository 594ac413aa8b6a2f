/* A stand-in for the CUDA runtime calls that lrscan's launches make, preloaded
 * by test_launch_cpu.py: it launches nothing, counts what it is asked for, and
 * keeps to the rules that the tests are about (attributes belong to a device; a
 * launch succeeds or fails by itself, whatever error an earlier call left). */
#include <stddef.h>

typedef struct { unsigned x, y, z; } Dim3;
typedef struct { Dim3 grid, block; size_t smem; void *stream, *attrs; unsigned n_attrs; } Config;

enum { MAX = 512, INVALID_VALUE = 1 };
static int device, pending, launches, fail_next, fail_attribute;
static struct { int dev; const void *func; size_t limit; } limits[MAX];
static int n_limits;

void fake_set_device(int d) { device = d; }
void fake_set_pending_error(int e) { pending = e; }
void fake_fail_next_launch(int n) { fail_next = n; }   /* the n-th from now */
void fake_fail_next_attribute(void) { fail_attribute = 1; }
int fake_launches(void) { return launches; }

int cudaGetDevice(int *d) { *d = device; return 0; }
int cudaDeviceGetAttribute(int *v, int attr, int dev) { (void)attr, (void)dev; *v = 152; return 0; }
int cudaGetLastError(void) { int e = pending; pending = 0; return e; }

int cudaFuncSetAttribute(const void *func, int attr, int value) {
    if (attr != 8 || n_limits == MAX || fail_attribute) {   /* MaxDynamicSharedMemorySize */
        fail_attribute = 0;
        return INVALID_VALUE;
    }
    limits[n_limits].dev = device, limits[n_limits].func = func, limits[n_limits].limit = (size_t)value;
    ++n_limits;
    return 0;
}

static int launch(const void *func, size_t smem) {
    size_t limit = 48 * 1024;
    for (int i = 0; i < n_limits; ++i)
        if (limits[i].dev == device && limits[i].func == func) limit = limits[i].limit;
    if (smem > limit || (fail_next > 0 && --fail_next == 0)) return pending = INVALID_VALUE;
    ++launches;
    return 0;
}
int cudaLaunchKernelExC(const Config *c, const void *func, void **args) { (void)args; return launch(func, c->smem); }
int __cudaGetKernel(void **k, const void *func) { *k = (void *)func; return 0; }
int __cudaLaunchKernel(void *k, Dim3 grid, Dim3 block, void **args, size_t smem, void *stream) {
    (void)grid, (void)block, (void)args, (void)stream;
    return launch(k, smem);
}

int cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int *n, const void *func, int threads, size_t smem,
                                                           unsigned flags) {
    (void)func, (void)threads, (void)smem, (void)flags;
    *n = 2;
    return 0;
}

static int encode(void) { return 0; }
int cudaGetDriverEntryPointByVersion(const char *name, void **fn, unsigned version, unsigned long long flags,
                                     int *found) {
    (void)name, (void)version, (void)flags;
    *fn = (void *)encode;
    if (found) *found = 0;
    return 0;
}
