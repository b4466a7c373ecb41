/*
 * A plain C caller of a residual block's row operators: no Python, no PyTorch.
 * Device memory and the workspace come from the CUDA runtime.
 *
 * usage: block_from_c ROWS COLS DIR
 * Reads from DIR (raw little-endian files):
 *   x.bin, r.bin, dy.bin  ROWS*COLS bf16 bit patterns: a branch's output, the residual,
 *                         the gradient of the norm
 *   gamma.bin             COLS fp32
 *   rng.bin               two int64: seed, offset
 * Writes to DIR: h.bin, y.bin (bf16), rstd.bin (fp32 [ROWS]) of fr_rmsnorm with dropout
 * 0.25 at site 7; q.bin (e4m3 bytes), scale.bin (fp32, one a row) of fr_rmsnorm_quant of h;
 * dx.bin, dres.bin (bf16), dgamma.bin (fp32 [COLS]) of fr_rmsnorm_backward with dh = dy;
 * drop.bin (bf16), fr_dropout of dres.  A short workspace, an output over another
 * one and dropout without its generator are refused.
 * Exit status 0 on success; any unexpected library or CUDA error exits 1.
 */
#include <cuda_runtime_api.h>
#include <stdio.h>
#include <stdlib.h>

#include "fr.h"

static int fail(const char *what, int code) {
  fprintf(stderr, "%s failed: %d\n", what, code);
  return 1;
}

/* A file of DIR in a new device buffer; NULL on failure. */
static void *load(const char *dir, const char *name, size_t bytes) {
  char path[4096];
  snprintf(path, sizeof path, "%s/%s", dir, name);
  FILE *f = fopen(path, "rb");
  if (!f) return NULL;
  void *h = malloc(bytes), *d = NULL;
  size_t got = h ? fread(h, 1, bytes, f) : 0;
  fclose(f);
  if (got == bytes && cudaMalloc(&d, bytes) == cudaSuccess &&
      cudaMemcpy(d, h, bytes, cudaMemcpyHostToDevice) != cudaSuccess)
    d = NULL;
  free(h);
  return d;
}

static int save(const char *dir, const char *name, const void *d, size_t bytes, cudaStream_t s) {
  char path[4096];
  snprintf(path, sizeof path, "%s/%s", dir, name);
  void *h = malloc(bytes);
  FILE *f = fopen(path, "wb");
  int bad = !h || !f || cudaMemcpyAsync(h, d, bytes, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
            cudaStreamSynchronize(s) != cudaSuccess || fwrite(h, 1, bytes, f) != bytes;
  if (f) fclose(f);
  free(h);
  return bad;
}

static void *room(size_t bytes) {
  void *d = NULL;
  return cudaMalloc(&d, bytes) == cudaSuccess ? d : NULL;
}

int main(int argc, char **argv) {
  if (argc != 4) {
    fprintf(stderr, "usage: %s ROWS COLS DIR\n", argv[0]);
    return 2;
  }
  const int64_t rows = atoll(argv[1]), cols = atoll(argv[2]);
  const char *dir = argv[3];
  const size_t n = (size_t)rows * (size_t)cols, r4 = (size_t)rows * 4, c4 = (size_t)cols * 4;
  const float eps = 1e-5f, p = 0.25f;
  void *x = load(dir, "x.bin", 2 * n), *r = load(dir, "r.bin", 2 * n), *dy = load(dir, "dy.bin", 2 * n);
  float *gamma = load(dir, "gamma.bin", c4);
  int64_t *rng = load(dir, "rng.bin", 16);
  void *h = room(2 * n), *y = room(2 * n), *q = room(n), *dx = room(2 * n), *dres = room(2 * n);
  float *rstd = room(r4), *scale = room(r4), *dgamma = room(c4);
  if (!x || !r || !dy || !gamma || !rng || !h || !y || !q || !dx || !dres || !rstd || !scale || !dgamma)
    return fail("inputs and buffers", 0);
  cudaStream_t s;
  cudaError_t e;
  if ((e = cudaStreamCreate(&s))) return fail("cudaStreamCreate", (int)e);
  fr_stream_t fs = (fr_stream_t)s;
  fr_status st;

  st = fr_rmsnorm(x, r, gamma, h, h, rstd, rows, cols, cols, cols, cols, cols, eps, p, rng, 7, FR_BF16,
                  FR_FORM_AUTO, fs);
  if (st != FR_ERR_INVALID_ARG) return fail("one output over another not refused", (int)st);
  st = fr_rmsnorm(x, r, gamma, h, y, rstd, rows, cols, cols, cols, cols, cols, eps, p, NULL, 7, FR_BF16,
                  FR_FORM_AUTO, fs);
  if (st != FR_ERR_INVALID_ARG) return fail("dropout without a generator not refused", (int)st);
  st = fr_rmsnorm(x, r, gamma, h, y, rstd, rows, cols, cols, cols, cols, cols, eps, p, rng, 7, FR_BF16,
                  FR_FORM_AUTO, fs);
  if (st != FR_OK) return fail(fr_status_string(st), (int)st);
  if (save(dir, "h.bin", h, 2 * n, s) || save(dir, "y.bin", y, 2 * n, s) ||
      save(dir, "rstd.bin", rstd, r4, s))
    return fail("fr_rmsnorm out", 0);

  st = fr_rmsnorm_quant(h, NULL, gamma, NULL, q, scale, FR_SCALE_ROW, 1, 1, NULL, rows, cols, cols, 0, 0,
                        cols, eps, 0.0f, NULL, 0, FR_BF16, FR_FORM_AUTO, fs);
  if (st != FR_OK) return fail(fr_status_string(st), (int)st);
  if (save(dir, "q.bin", q, n, s) || save(dir, "scale.bin", scale, r4, s))
    return fail("fr_rmsnorm_quant out", 0);

  const size_t ws = fr_workspace_size(FR_OP_RMSNORM_BACKWARD, rows, cols, FR_BF16, FR_FORM_AUTO);
  void *w = ws ? room(ws) : NULL;
  if (!w) return fail("workspace", (int)ws);
  for (int k = 0; k < 2; ++k) {
    st = fr_rmsnorm_backward(dy, h, gamma, rstd, dy, dx, dres, dgamma, rows, cols, cols, cols, cols, cols,
                             cols, p, rng, 7, FR_BF16, FR_FORM_AUTO, w, k ? ws : ws - 1, fs);
    if (st != (k ? FR_OK : FR_ERR_WORKSPACE_TOO_SMALL)) return fail("fr_rmsnorm_backward", (int)st);
  }
  if (save(dir, "dx.bin", dx, 2 * n, s) || save(dir, "dres.bin", dres, 2 * n, s) ||
      save(dir, "dgamma.bin", dgamma, c4, s))
    return fail("fr_rmsnorm_backward out", 0);

  st = fr_dropout(dres, NULL, dres, rows, cols, cols, 0, cols, p, rng, 7, FR_BF16, fs);
  if (st != FR_OK) return fail(fr_status_string(st), (int)st);
  if (save(dir, "drop.bin", dres, 2 * n, s)) return fail("fr_dropout out", 0);

  int32_t code = -1;
  if (fr_check_device_error(fs, &code) != FR_OK) return fail("device error", (int)code);
  void *bufs[] = {x, r, dy, gamma, rng, h, y, q, dx, dres, rstd, scale, dgamma, w};
  for (size_t k = 0; k < sizeof bufs / sizeof bufs[0]; ++k) cudaFree(bufs[k]);
  cudaStreamDestroy(s);
  return 0;
}
