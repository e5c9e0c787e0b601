/* A stand-in for the HIP runtime that only writes down what is launched: opened with
 * global symbols before liblogra.so, it is what the library's kernels are registered
 * with and launched through, so that accepted calls can be followed on a machine without a
 * GPU.  Nothing is run and no pointer is looked at.
 */
#include <stddef.h>
#include <stdint.h>
#include <string.h>

typedef struct {
  uint32_t x, y, z;
} dim3_t;

typedef struct {
  const char* name;    /* as registered (mangled) */
  uint32_t grid[3], block[3];
} launch_t;

#define MAX_KERNELS 4096
#define MAX_LAUNCHES 4096
static struct {
  const void* stub;
  const char* name;
} g_kernels[MAX_KERNELS];
static int g_n_kernels;
static launch_t g_launches[MAX_LAUNCHES];
static int g_n_launches;
static dim3_t g_grid, g_block;
static size_t g_lds;
static void* g_stream;

int fake_hip_kernels(void) { return g_n_kernels; }
void fake_hip_clear(void) { g_n_launches = 0; }
int fake_hip_launches(void) { return g_n_launches; }
const launch_t* fake_hip_launch(int i) { return &g_launches[i]; }

static void* g_module;
void** __hipRegisterFatBinary(const void* data) {
  (void)data;
  return &g_module;
}
void __hipUnregisterFatBinary(void** modules) { (void)modules; }
void __hipRegisterFunction(void** modules, const void* stub, char* name, const char* device_name,
                           unsigned limit, void* tid, void* bid, dim3_t* block, dim3_t* grid,
                           int* wave) {
  (void)modules, (void)device_name, (void)limit, (void)tid, (void)bid, (void)block, (void)grid,
      (void)wave;
  if (g_n_kernels < MAX_KERNELS) {
    g_kernels[g_n_kernels].stub = stub;
    g_kernels[g_n_kernels++].name = name;
  }
}
int __hipPushCallConfiguration(dim3_t grid, dim3_t block, size_t lds, void* stream) {
  g_grid = grid, g_block = block, g_lds = lds, g_stream = stream;
  return 0;
}
int __hipPopCallConfiguration(dim3_t* grid, dim3_t* block, size_t* lds, void** stream) {
  *grid = g_grid, *block = g_block, *lds = g_lds, *stream = g_stream;
  return 0;
}
int hipLaunchKernel(const void* stub, dim3_t grid, dim3_t block, void** args, size_t lds,
                    void* stream) {
  (void)args, (void)lds, (void)stream;
  if (g_n_launches == MAX_LAUNCHES) return 1;
  launch_t* const l = &g_launches[g_n_launches++];
  l->name = "?";
  for (int i = 0; i < g_n_kernels; ++i)
    if (g_kernels[i].stub == stub) l->name = g_kernels[i].name;
  memcpy(l->grid, &grid, sizeof(grid));
  memcpy(l->block, &block, sizeof(block));
  return 0;
}
int hipGetLastError(void) { return 0; }
int hipPeekAtLastError(void) { return 0; }
void __hipRegisterVar(void** modules, void* var, char* name, char* device_name, int ext, size_t size,
                      int constant, int global) {
  (void)modules, (void)var, (void)name, (void)device_name, (void)ext, (void)size, (void)constant,
      (void)global;
}
int hipGetDevice(int* device) {
  *device = 0;
  return 0;
}
int hipSetDevice(int device) { return device != 0; }
int hipStreamGetDevice(void* stream, int* device) {
  (void)stream;
  *device = 0;
  return 0;
}
int hipGetSymbolAddress(void** at, const void* symbol) {
  (void)symbol;
  *at = NULL;
  return 1;
}
const char* hipGetErrorString(int error) {
  (void)error;
  return "";
}
