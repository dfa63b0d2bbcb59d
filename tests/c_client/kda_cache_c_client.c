/*
 * A plain C99 client of the cache and beam entry points: it takes each by
 * address, computes rotation steps, asks for workspace sizes, and checks that
 * malformed calls are refused with a message before any CUDA work.  It needs
 * no GPU.  Exit status 0 when every check holds.
 */
#include <stdio.h>
#include <string.h>

#include "kda.h"

static int failures = 0;

static void expect(int ok, const char* what) {
  if (!ok) {
    fprintf(stderr, "FAILED: %s (%s)\n", what, kda_last_error_message());
    ++failures;
  }
}

typedef void (*any_fn)(void);

int main(void) {
  const any_fn fns[] = {(any_fn)kda_rope_append, (any_fn)kda_rope_phase_steps, (any_fn)kda_paged_attention_decode,
                        (any_fn)kda_paged_attention_workspace, (any_fn)kda_beam_select,
                        (any_fn)kda_beam_select_workspace, (any_fn)kda_pool_move};
  size_t i;
  for (i = 0; i < sizeof(fns) / sizeof(fns[0]); ++i) expect(fns[i] != NULL, "declared function resolves");

  {
    uint64_t steps[32];
    int64_t floats = 0;
    expect(kda_rope_phase_steps(64, 10000.0, 1.0, 0.0, 1.0, 32.0, steps) == KDA_OK, "rotation steps");
    /* the first pair turns by one radian a position: 2^64 / 2 pi */
    expect(steps[0] > 2935890503282001000ull && steps[0] < 2935890503282002000ull, "one radian a position");
    for (i = 1; i < 32; ++i) expect(steps[i] < steps[i - 1], "falling frequencies");
    expect(kda_rope_phase_steps(7, 10000.0, 1.0, 0.0, 1.0, 32.0, steps) == KDA_ERR_INVALID_ARG, "odd rotated part");
    expect(kda_rope_phase_steps(64, 10000.0, 1.0, 0.0, 1.0, 32.0, NULL) == KDA_ERR_INVALID_ARG, "null steps");
    expect(kda_paged_attention_workspace(32, 8, 128, KDA_BF16, 152, &floats) == KDA_OK && floats > 0, "attention workspace");
    expect(kda_paged_attention_workspace(32, 7, 128, KDA_BF16, 152, &floats) == KDA_ERR_INVALID_ARG, "uneven heads");
    expect(kda_paged_attention_workspace(32, 8, 100, KDA_BF16, 152, &floats) == KDA_ERR_UNSUPPORTED, "head dimension");
    expect(kda_beam_select_workspace(4, 4, 32000, 8, KDA_F32, 152, &floats) == KDA_OK && floats > 0, "beam workspace");
    expect(kda_beam_select_workspace(4, 40, 32000, 8, KDA_F32, 152, &floats) == KDA_ERR_UNSUPPORTED, "too many beams");
  }
  {
    kda_tensor t;
    const kda_tensor* p = &t;
    memset(&t, 0, sizeof(t));
    expect(kda_rope_append(NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, 0, 1.f, NULL) == KDA_ERR_INVALID_ARG,
           "rope: null descriptors");
    expect(kda_rope_append(p, p, p, p, p, p, p, p, p, p, 0, 1.f, NULL) == KDA_ERR_INVALID_ARG, "rope: rank 0");
    expect(kda_paged_attention_decode(p, p, p, p, p, p, 0, 0.1f, p, p, NULL) == KDA_ERR_INVALID_ARG, "attention: rank 0");
    expect(kda_beam_select(p, p, p, 0, p, p, p, p, NULL) == KDA_ERR_INVALID_ARG, "beam: rank 0");
    expect(kda_pool_move(&p, 1, p, p, NULL, NULL) == KDA_ERR_INVALID_ARG, "move: rank 0");
    expect(kda_pool_move(NULL, 1, p, p, NULL, NULL) == KDA_ERR_INVALID_ARG, "move: null pools");
    expect(kda_pool_move(&p, 0, p, p, NULL, NULL) == KDA_ERR_INVALID_ARG, "move: no pools");
    expect(strlen(kda_last_error_message()) > 0, "message");
  }
  if (failures != 0) return 1;
  printf("all checks passed\n");
  return 0;
}
