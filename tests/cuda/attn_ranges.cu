// Host build of the attention kernels' range arithmetic (attn_seq, add_items), so that it can
// be checked for every kind of caller's numbers without a GPU.
#include "../../packed_linear_attention_gb300/csrc/gdn_attn_internal.h"

extern "C" void attn_ranges(int num_seqs, int num_tokens, int max_q_len, int max_kv_len,
                            int max_blocks, int page_size, const int* cu_q, const int* kv_len,
                            int* row0, int* q_len, int* kv, int* bad) {
  gdn::AttnArgs a = {};
  a.cu_q = cu_q;
  a.kv_len = kv_len;
  a.num_seqs = num_seqs;
  a.num_tokens = num_tokens;
  a.max_q_len = max_q_len;
  a.max_kv_len = max_kv_len;
  a.max_blocks = max_blocks;
  a.page_size = page_size;
  for (int b = 0; b < num_seqs; ++b) {
    bool cut = false;
    const gdn::AttnSeq s = gdn::attn_seq(a, b, cut);
    row0[b] = s.row0;
    q_len[b] = s.q_len;
    kv[b] = s.kv_len;
    bad[b] = cut;
  }
}

extern "C" int attn_items_sum(int n, const int* items) {
  int sum = 0;
  for (int i = 0; i < n; ++i) sum = gdn::add_items(sum, items[i]);
  return sum;
}
