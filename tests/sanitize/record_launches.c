// Preloaded in front of the HIP runtime: writes down every kernel launch's
// grid and block, and launches nothing.  (dim3 as the runtime passes it.)
#include <stddef.h>
#include <stdio.h>
#include <stdlib.h>

typedef struct {
  unsigned x, y, z;
} dim3;

static struct {
  dim3 grid, block;
  size_t lds;
  void* stream;
} now;

int __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, void* stream) {
  now.grid = grid, now.block = block, now.lds = lds, now.stream = stream;
  return 0;
}
int __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, void** stream) {
  *grid = now.grid, *block = now.block, *lds = now.lds, *stream = now.stream;
  return 0;
}
int hipLaunchKernel(const void* kernel, dim3 grid, dim3 block, void** args, size_t lds, void* stream) {
  (void)kernel, (void)args, (void)lds, (void)stream;
  FILE* f = fopen(getenv("SEED_LAUNCHES"), "a");
  if (!f) return 1;
  fprintf(f, "%u %u %u %u %u %u\n", grid.x, grid.y, grid.z, block.x, block.y, block.z);
  fclose(f);
  return 0;
}
int hipFuncSetAttribute(const void* kernel, int attribute, int value) {
  (void)kernel, (void)attribute, (void)value;
  return 0;
}
int hipGetLastError(void) { return 0; }
