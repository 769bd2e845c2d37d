/* The CUDA runtime's calls that the tree operators' host side makes, without a
 * GPU: each is noted in a log, device memory is the host's, launches do nothing.
 * The current device is what cudaSetDevice said. */
#include <stdarg.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

static char text[1 << 16];
static size_t used;
static int current;

static int note(const char *format, ...) {
  va_list a;
  va_start(a, format);
  if (used < sizeof text - 200) used += vsnprintf(text + used, 200, format, a);
  va_end(a);
  return 0;
}

const char *fake_log(void) { return text; }
void fake_clear(void) { used = 0, text[0] = 0; }

int cudaGetDevice(int *d) { return *d = current, 0; }
int cudaSetDevice(int d) { return current = d, note("device %d\n", d); }
int cudaDeviceGetAttribute(int *value, int attr, int device) {
  (void)device;
  *value = attr == 75 ? 10 : attr == 76 ? 3 : attr == 16 ? 152 : 0; /* capability, SMs */
  return 0;
}
int cudaMalloc(void **p, size_t n) {
  *p = aligned_alloc(256, (n + 255) / 256 * 256);
  memset(*p, 0x5a, n);
  return note("malloc on %d\n", current);
}
int cudaFree(void *p) { return free(p), note("free on %d\n", current); }
int cudaMemset(void *p, int v, size_t n) {
  return memset(p, v, n), note("memset stream 0 on %d\n", current);
}
int cudaMemsetAsync(void *p, int v, size_t n, void *s) {
  return memset(p, v, n), note("memset stream %p on %d\n", s, current);
}
int cudaMemcpyAsync(void *d, const void *p, size_t n, int kind, void *s) {
  (void)kind;
  return memcpy(d, p, n), note("copy stream %p on %d\n", s, current);
}
int cudaStreamCreateWithFlags(void **s, unsigned flags) {
  *s = (void *)0x77;
  return note("stream %p flags %u on %d\n", *s, flags, current);
}
int cudaStreamDestroy(void *s) { return note("destroy stream %p on %d\n", s, current); }
int cudaStreamSynchronize(void *s) { return note("synchronise stream %p on %d\n", s, current); }
int cudaDeviceSynchronize(void) { return note("synchronise all on %d\n", current); }
int cudaGetDriverEntryPointByVersion(const char *name, void **f, unsigned v, unsigned long long flags,
                                     int *found) {
  (void)name, (void)v, (void)flags;
  *f = 0, *found = 1;
  return 0;
}
int cudaFuncSetAttribute(const void *f, int attr, int value) {
  (void)f, (void)attr, (void)value;
  return 0;
}
int cudaGetLastError(void) { return 0; }
int cudaLaunchKernelExC(const void *config, const void *f, void **args) {
  (void)config, (void)f, (void)args;
  return note("launch on %d\n", current);
}
typedef struct { unsigned x, y, z; } dim3;
/* what the compiler makes of <<< >>> */
int __cudaGetKernel(void **kernel, const void *f) { return *kernel = (void *)f, 0; }
int __cudaLaunchKernel(void *kernel, dim3 grid, dim3 block, void **args, size_t smem, void *s) {
  (void)kernel, (void)args, (void)smem, (void)s;
  return note("launch grid %u %u %u block %u on %d\n", grid.x, grid.y, grid.z, block.x, current);
}
