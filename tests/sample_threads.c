/* Calls of confkv_sample from several threads at once, each with its own row
 * size and stream. Built and called by tests/test_gpu_sample.py. */
#include <pthread.h>
#include <stddef.h>

#include "confkv.h"

typedef confkv_status (*sample_fn)(int32_t, const void*, int64_t, int32_t, int32_t, const float*, const float*,
                                   const int32_t*, const float*, const float*, int32_t*, float*, void*);

typedef struct {
  const float* logits;
  int32_t rows, vocab;
  const float *u, *top_p;
  int32_t* token;
  void* stream;
  int32_t calls;
  int32_t failed; /* out: calls that did not return CONFKV_OK */
  sample_fn sample;
} job;

static void* run(void* p) {
  job* j = (job*)p;
  for (int32_t i = 0; i < j->calls; ++i)
    if (j->sample(CONFKV_F32, j->logits, j->vocab, j->rows, j->vocab, j->u, NULL, NULL, j->top_p, NULL, j->token, NULL,
                  j->stream) != CONFKV_OK)
      ++j->failed;
  return NULL;
}

/* Returns 0 once every thread has run, whatever its calls returned. */
int run_threads(job* jobs, int n) {
  pthread_t t[16];
  int started = 0, rc = 0;
  if (n < 1 || n > 16) return 1;
  for (; started < n; ++started)
    if (pthread_create(&t[started], NULL, run, &jobs[started]) != 0) {
      rc = 2;
      break;
    }
  for (int i = 0; i < started; ++i) pthread_join(t[i], NULL);
  return rc;
}
