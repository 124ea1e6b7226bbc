/* The HIP launch interface as a recorder: loaded with global symbols before libfluxbin.so, it takes the
 * library's kernel registrations and launches, so that the host side of an entry point (checks, choice of
 * a kernel, grid, arguments) can be watched without a GPU.  Nothing is run. */
#include <stddef.h>
#include <stdint.h>
#include <string.h>

typedef struct { uint32_t x, y, z; } dim;
typedef struct { const char *kernel; dim grid, block; uint8_t args[256]; } launch;

enum { KERNELS = 4096, LAUNCHES = 4096 };
static struct { const void *host; const char *name; } kernels[KERNELS];
static int n_kernels, n_launches;
static launch launches[LAUNCHES];
static dim next_grid, next_block;

void **__hipRegisterFatBinary(const void *data) {
  static void *handle;
  (void)data;
  return &handle;
}
void __hipUnregisterFatBinary(void **handle) { (void)handle; }
void __hipRegisterVar(void **handle, void *var, char *host, char *dev, int ext, size_t size, int constant, int global) {
  (void)handle, (void)var, (void)host, (void)dev, (void)ext, (void)size, (void)constant, (void)global;
}
void __hipRegisterFunction(void **handle, const void *host, char *dev, const char *name, unsigned limit, void *tid, void *bid,
                           void *block, void *grid, int *wsize) {
  (void)handle, (void)dev, (void)limit, (void)tid, (void)bid, (void)block, (void)grid, (void)wsize;
  if (n_kernels < KERNELS) {
    kernels[n_kernels].host = host;
    kernels[n_kernels++].name = name;
  }
}
int __hipPushCallConfiguration(dim grid, dim block, size_t shared, void *stream) {
  (void)shared, (void)stream;
  next_grid = grid;
  next_block = block;
  return 0;
}
int __hipPopCallConfiguration(dim *grid, dim *block, size_t *shared, void **stream) {
  *grid = next_grid;
  *block = next_block;
  *shared = 0;
  *stream = NULL;
  return 0;
}
/* args[0]: the kernel's one argument, a struct whose size the reader knows (at most 256 bytes are kept). */
static size_t arg_bytes = 0;
int hipLaunchKernel(const void *host, dim grid, dim block, void **args, size_t shared, void *stream) {
  (void)shared, (void)stream;
  if (n_launches == LAUNCHES) return 1;
  launch *l = &launches[n_launches++];
  l->kernel = "?";
  for (int i = 0; i < n_kernels; ++i)
    if (kernels[i].host == host) l->kernel = kernels[i].name;
  l->grid = grid;
  l->block = block;
  if (arg_bytes <= sizeof l->args) memcpy(l->args, args[0], arg_bytes);
  return 0;
}
int hipGetLastError(void) { return 0; }

void recorder_start(size_t bytes) {
  n_launches = 0;
  arg_bytes = bytes;
}
int recorder_count(void) { return n_launches; }
const launch *recorder_launch(int i) { return &launches[i]; }
int recorder_kernels(void) { return n_kernels; }
const char *recorder_kernel(int i) { return kernels[i].name; }
