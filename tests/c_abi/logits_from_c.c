/*
 * A plain C caller of the entry points for rows of logits: no Python, no
 * PyTorch.  Device memory and the workspace come from the CUDA runtime.
 *
 * usage: logits_from_c ROWS COLS TOP DIR
 * Reads from DIR (raw little-endian files):
 *   x.bin   ROWS*COLS bf16 bit patterns      t.bin   ROWS int64 tokens
 *   i.bin   ROWS*TOP int64 teacher indices   z.bin   ROWS*TOP fp32 teacher logits
 *   g.bin   ROWS fp32 upstream gradients
 * Writes to DIR: logprob.bin, entropy.bin, lse.bin, loss.bin (fr_xent_backward's),
 * distill.bin, distill_step.bin (fr_distill's and fr_distill_backward's losses; all
 * fp32 [ROWS]), top.bin (int64 [ROWS, TOP]), xent.bin, distill_grad.bin,
 * logprobs_grad.bin (bf16 [ROWS, COLS]; the last in place over the logits, from both
 * upstream gradients being g.bin).  fr_logprobs runs in the looped form, whose
 * alternatives need the workspace; a short workspace and a missing one are refused.
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
  if (argc != 5) {
    fprintf(stderr, "usage: %s ROWS COLS TOP DIR\n", argv[0]);
    return 2;
  }
  const int64_t rows = atoll(argv[1]), cols = atoll(argv[2]);
  const int32_t top = atoi(argv[3]);
  const char *dir = argv[4];
  const size_t n = (size_t)rows * (size_t)cols * 2, nt = (size_t)rows * (size_t)top;
  void *x = load(dir, "x.bin", n);
  int64_t *t = load(dir, "t.bin", (size_t)rows * 8), *i = load(dir, "i.bin", nt * 8);
  float *z = load(dir, "z.bin", nt * 4), *g = load(dir, "g.bin", (size_t)rows * 4);
  float *logprob = room((size_t)rows * 4), *entropy = room((size_t)rows * 4),
        *lse = room((size_t)rows * 4), *loss = room((size_t)rows * 4), *tl = room(nt * 4);
  int64_t *ti = room(nt * 8);
  void *d = room(n);
  if (!x || !t || !i || !z || !g || !logprob || !entropy || !lse || !loss || !tl || !ti || !d)
    return fail("inputs and buffers", 0);
  cudaStream_t s;
  cudaError_t e;
  if ((e = cudaStreamCreate(&s))) return fail("cudaStreamCreate", (int)e);
  fr_stream_t fs = (fr_stream_t)s;
  fr_status st;

  const size_t ws = fr_workspace_size(FR_OP_LOGPROBS, rows, cols, FR_BF16, FR_FORM_LOOPED);
  void *w = ws ? room(ws) : NULL;
  if (!w) return fail("workspace", (int)ws);
  st = fr_logprobs(x, t, logprob, entropy, lse, tl, ti, top, rows, cols, cols, -100, FR_BF16,
                   FR_FORM_LOOPED, w, ws - 1, fs);
  if (st != FR_ERR_WORKSPACE_TOO_SMALL) return fail("short workspace not refused", (int)st);
  st = fr_logprobs(x, t, logprob, entropy, lse, tl, ti, top, rows, cols, cols, -100, FR_BF16,
                   FR_FORM_LOOPED, NULL, 0, fs);
  if (st != FR_ERR_WORKSPACE_TOO_SMALL) return fail("missing workspace not refused", (int)st);
  st = fr_logprobs(x, t, logprob, entropy, lse, tl, ti, top, rows, cols, cols, -100, FR_BF16,
                   FR_FORM_LOOPED, w, ws, fs);
  if (st != FR_OK) return fail(fr_status_string(st), (int)st);
  if (fr_last_form() != FR_FORM_LOOPED) return fail("form", (int)fr_last_form());
  if (save(dir, "logprob.bin", logprob, (size_t)rows * 4, s) ||
      save(dir, "entropy.bin", entropy, (size_t)rows * 4, s) ||
      save(dir, "lse.bin", lse, (size_t)rows * 4, s) || save(dir, "top.bin", ti, nt * 8, s))
    return fail("fr_logprobs out", 0);

  st = fr_xent_backward(x, t, g, 1, loss, d, rows, cols, cols, cols, -100, FR_BF16, FR_FORM_AUTO,
                        fs);
  if (st != FR_OK) return fail(fr_status_string(st), (int)st);
  if (save(dir, "loss.bin", loss, (size_t)rows * 4, s) || save(dir, "xent.bin", d, n, s))
    return fail("fr_xent_backward out", 0);

  st = fr_distill(x, i, z, loss, top, rows, cols, cols, top, 2.0f, FR_BF16, FR_FORM_AUTO, fs);
  if (st != FR_OK) return fail(fr_status_string(st), (int)st);
  if (save(dir, "distill.bin", loss, (size_t)rows * 4, s)) return fail("fr_distill out", 0);
  st = fr_distill_backward(x, i, z, g, 1, loss, d, top, rows, cols, cols, cols, top, 2.0f, FR_BF16,
                           FR_FORM_AUTO, fs);
  if (st != FR_OK) return fail(fr_status_string(st), (int)st);
  if (save(dir, "distill_step.bin", loss, (size_t)rows * 4, s) ||
      save(dir, "distill_grad.bin", d, n, s))
    return fail("fr_distill_backward out", 0);

  st = fr_logprobs_backward(x, t, g, 1, g, 1, x, rows, cols, cols, cols, -100, FR_BF16,
                            FR_FORM_AUTO, fs);
  if (st != FR_OK) return fail(fr_status_string(st), (int)st);
  if (save(dir, "logprobs_grad.bin", x, n, s)) return fail("fr_logprobs_backward out", 0);

  int32_t code = -1;
  if (fr_check_device_error(fs, &code) != FR_OK) return fail("device error", (int)code);
  void *bufs[] = {x, t, i, z, g, logprob, entropy, lse, loss, tl, ti, d, w};
  for (size_t k = 0; k < sizeof bufs / sizeof bufs[0]; ++k) cudaFree(bufs[k]);
  cudaStreamDestroy(s);
  return 0;
}
