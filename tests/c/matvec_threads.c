/* Products from codes by several host threads at once, each on a stream of its own: rows of an odd
 * width, whose x is laid out in shared memory, of another size in each thread, by one and the same
 * kernel. Every call has to succeed and every result has to be the one of a lone call. Exit
 * status 0 on success. */
#include <pthread.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
#include <cuda_runtime_api.h>
#include "zpp.h"

enum { THREADS = 4, ROWS = 8, VECS = 8, BLOCK = 64, CALLS = 5000 };
static const long long kCols[THREADS] = {40001, 12001, 24001, 60001};

struct job {
  long long cols;
  void *codes, *x;
  float *scales, *y;
  float want[VECS * ROWS];
  cudaStream_t stream;
  int failed, first;
};
static pthread_barrier_t start;

static int product(struct job* j) {
  return zpp_matvec_blockwise(j->codes, j->scales, ROWS, j->cols, BLOCK, 4, j->x, ZPP_F16, VECS, j->cols,
                              NULL, j->y, ZPP_F32, ROWS, j->stream);
}

static void* work(void* p) {
  struct job* j = p;
  pthread_barrier_wait(&start);
  for (int i = 0; i < CALLS; ++i) {
    const int status = product(j);
    if (status != ZPP_OK && j->failed++ == 0) j->first = status;
  }
  return NULL;
}

#define TRY(e)                                       \
  do {                                               \
    if ((e) != cudaSuccess) {                        \
      fprintf(stderr, "FAILED: %s\n", #e);           \
      return 1;                                      \
    }                                                \
  } while (0)

int main(void) {
  static struct job jobs[THREADS];
  float got[VECS * ROWS];
  for (int t = 0; t < THREADS; ++t) {
    struct job* j = &jobs[t];
    j->cols = kCols[t];
    const size_t n = (size_t)(ROWS * j->cols), blocks = (n + BLOCK - 1) / BLOCK, xs = (size_t)(VECS * j->cols);
    unsigned char* codes = malloc((n + 1) / 2);
    unsigned short* x = malloc(xs * 2);
    float* scales = malloc(blocks * 4);
    for (size_t i = 0; i < (n + 1) / 2; ++i) codes[i] = (unsigned char)((i * 7 % 7) | (i * 5 % 7) << 4);
    for (size_t i = 0; i < xs; ++i) x[i] = i % 3 == 0 ? 0x3c00 : 0; /* 1 or 0 */
    for (size_t i = 0; i < blocks; ++i) scales[i] = i % 2 ? 1.0f : 0.5f;
    TRY(cudaMalloc(&j->codes, (n + 1) / 2));
    TRY(cudaMalloc((void**)&j->scales, blocks * 4));
    TRY(cudaMalloc(&j->x, xs * 2));
    TRY(cudaMalloc((void**)&j->y, sizeof got));
    TRY(cudaMemcpy(j->codes, codes, (n + 1) / 2, cudaMemcpyHostToDevice));
    TRY(cudaMemcpy(j->scales, scales, blocks * 4, cudaMemcpyHostToDevice));
    TRY(cudaMemcpy(j->x, x, xs * 2, cudaMemcpyHostToDevice));
    TRY(cudaStreamCreateWithFlags(&j->stream, cudaStreamNonBlocking));
    free(codes), free(x), free(scales);
    if (product(j) != ZPP_OK) {
      fprintf(stderr, "FAILED: a lone call\n");
      return 1;
    }
    TRY(cudaStreamSynchronize(j->stream));
    TRY(cudaMemcpy(j->want, j->y, sizeof got, cudaMemcpyDeviceToHost));
  }
  pthread_t threads[THREADS];
  pthread_barrier_init(&start, NULL, THREADS);
  for (int t = 0; t < THREADS; ++t) pthread_create(&threads[t], NULL, work, &jobs[t]);
  for (int t = 0; t < THREADS; ++t) pthread_join(threads[t], NULL);
  int bad = 0;
  for (int t = 0; t < THREADS; ++t) {
    TRY(cudaStreamSynchronize(jobs[t].stream));
    TRY(cudaMemcpy(got, jobs[t].y, sizeof got, cudaMemcpyDeviceToHost));
    if (jobs[t].failed || memcmp(got, jobs[t].want, sizeof got)) {
      fprintf(stderr, "FAILED: thread %d, %d of %d calls refused (first status %d)\n", t, jobs[t].failed,
              CALLS, jobs[t].first);
      bad = 1;
    }
  }
  if (!bad) printf("threads OK\n");
  return bad;
}
