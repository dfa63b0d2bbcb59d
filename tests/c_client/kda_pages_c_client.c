/*
 * A plain C99 client of page assignment, rotary positions with several axes and
 * shared-prefix attention: it takes each by address, lays out pair axes, asks
 * for a workspace, and checks that malformed calls are refused with a message
 * before any CUDA work.  It needs no GPU.  Exit status 0 when every check holds.
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
  const any_fn fns[] = {(any_fn)kda_page_assign, (any_fn)kda_rope_axes_append, (any_fn)kda_rope_pair_axes,
                        (any_fn)kda_prefix_attention_decode, (any_fn)kda_prefix_attention_workspace};
  size_t i;
  for (i = 0; i < sizeof(fns) / sizeof(fns[0]); ++i) expect(fns[i] != NULL, "declared function resolves");

  {
    const int32_t sections[3] = {2, 3, 1}, bad[2] = {1, -1};
    const int32_t want[6] = {0, 1, 2, 0, 1, 1};
    int32_t axes[6];
    int64_t floats = 0;
    expect(kda_rope_pair_axes(sections, 3, 1, axes) == KDA_OK && memcmp(axes, want, sizeof(want)) == 0, "axes in turn");
    expect(kda_rope_pair_axes(bad, 2, 0, axes) == KDA_ERR_INVALID_ARG, "negative section");
    expect(kda_rope_pair_axes(sections, 5, 0, axes) == KDA_ERR_UNSUPPORTED, "too many axes");
    expect(kda_rope_pair_axes(sections, 3, 2, axes) == KDA_ERR_INVALID_ARG, "cyclic is 0 or 1");
    expect(kda_rope_pair_axes(NULL, 3, 0, axes) == KDA_ERR_INVALID_ARG, "null sections");
    expect(kda_rope_pair_axes(sections, 3, 0, NULL) == KDA_ERR_INVALID_ARG, "null axes");
    expect(kda_prefix_attention_workspace(64, 32, 8, 128, KDA_BF16, 152, &floats) == KDA_OK && floats > 0, "workspace");
    expect(kda_prefix_attention_workspace(-1, 32, 8, 128, KDA_BF16, 152, &floats) == KDA_ERR_UNSUPPORTED, "negative count");
    expect(kda_prefix_attention_workspace(64, 32, 7, 128, KDA_BF16, 152, &floats) == KDA_ERR_INVALID_ARG, "uneven heads");
    expect(kda_prefix_attention_workspace(64, 32, 8, 128, KDA_BF16, 152, NULL) == KDA_ERR_INVALID_ARG, "null floats");
  }
  {
    kda_tensor t;
    const kda_tensor* p = &t;
    memset(&t, 0, sizeof(t));
    expect(kda_page_assign(NULL, NULL, NULL, NULL, NULL, NULL, 16, NULL, NULL, NULL, NULL, NULL) == KDA_ERR_INVALID_ARG,
           "pages: null descriptors");
    expect(kda_page_assign(p, p, NULL, p, p, p, 16, p, p, p, p, NULL) == KDA_ERR_INVALID_ARG, "pages: rank 0");
    expect(kda_rope_axes_append(p, p, p, p, p, p, p, p, p, p, 0, 1.f, NULL) == KDA_ERR_INVALID_ARG, "axes: rank 0");
    expect(kda_prefix_attention_decode(p, p, p, p, p, p, p, p, 0, 0.1f, p, p, NULL) == KDA_ERR_INVALID_ARG, "prefix: rank 0");
    expect(strlen(kda_last_error_message()) > 0, "message");
  }
  if (failures != 0) return 1;
  printf("all checks passed\n");
  return 0;
}
