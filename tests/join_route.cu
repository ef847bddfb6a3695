// Which kernels the entry points of attention choose, on the host: the library's
// own checks and plans, with launches that note their names.
//
// stdin: calls of "diff e4m3 D q_heads kv_heads page causal window nk max_q
// total_q batch groups max_prefix max_own max_group" (groups 0: nothing shared).
// stdout, for each: the status, then the passes' kernels in the order of their
// launches ("prefix:chunk own:tokens"; one launch of two is "both:tokens").
#include <cstdio>
#include <string>

#include "santa_paged_api.cu"

static std::string got;

namespace santa {

static cudaError_t note(const char* kernel, const JoinArgs* first, const JoinArgs& a) {
  got += std::string(first ? " both:" : a.phase == 1 ? " prefix:" : " own:") + kernel;
  return cudaSuccess;
}
static void few(PagedArgs& a, int rows) {
  a.rows = rows, a.tokens = 0, a.splits = 1, a.split_blk = 1 << 27;
  a.tiles = (int)(((long long)a.max_q * a.G + rows - 1) / rows);
}
size_t plan_paged_tokens(PagedArgs& a) { few(a, 16); return 0; }
int plan_paged_chunk(PagedArgs& a) { a.splits = a.num_sms, a.rows = 2 * CHUNK_ROWS; return 0; }
void plan_tokens(PagedArgs& a, int, int, int) { few(a, 16); }
void plan_diff_tokens(JoinArgs& a, int, int) { few(a, 8); }
cudaError_t launch_paged_tokens(const PagedArgs&) { got += " tokens"; return cudaSuccess; }
cudaError_t launch_paged_chunk(const PagedArgs&) { got += " chunk"; return cudaSuccess; }
cudaError_t launch_join_tokens(const JoinArgs* p, const JoinArgs& a, bool) { return note("tokens", p, a); }
cudaError_t launch_diff_tokens(const JoinArgs* p, const JoinArgs& a, bool) { return note("tokens", p, a); }
cudaError_t launch_join_chunk(const JoinArgs& a, bool) { return note("chunk", nullptr, a); }
cudaError_t launch_diff_chunk(const JoinArgs& a, bool) { return note("chunk", nullptr, a); }
cudaError_t launch_diff_wide(const JoinArgs& a, bool) { return note("wide", nullptr, a); }
cudaError_t launch_join(const JoinArgs&, const JoinArgs&) { return cudaSuccess; }
cudaError_t launch_kv_append(const PagedArgs&, const AppendArgs&) { return cudaSuccess; }
cudaError_t launch_kv_read(const PagedArgs&, const int64_t*, long long, void*, void*) { return cudaSuccess; }

}  // namespace santa

int main() {
  int diff, e4m3, D, H, Hkv, page, causal, window, max_q, batch, groups, max_group;
  long long nk, total_q, max_prefix, max_own;
  void* const at = reinterpret_cast<void*>(1ull << 32);   // never read
  while (std::scanf("%d %d %d %d %d %d %d %d %lld %d %lld %d %d %lld %lld %d", &diff, &e4m3, &D, &H, &Hkv, &page, &causal, &window, &nk,
                    &max_q, &total_q, &batch, &groups, &max_prefix, &max_own, &max_group) == 16) {
    santa_paged_t p = {};
    p.batch = batch, p.n_q_heads = H, p.n_kv_heads = Hkv, p.head_dim = D;
    p.dtype = SANTA_BF16, p.cache_dtype = e4m3 ? SANTA_E4M3 : SANTA_BF16;
    p.page_size = page, p.n_pages = 1 << 14, p.max_pages = (int)((nk + page - 1) / page);
    p.page_table = static_cast<int32_t*>(at), p.kv_lens = p.page_table, p.q_offsets = static_cast<int64_t*>(at);
    p.nk = nk, p.max_q = max_q, p.total_q = total_q, p.causal = causal, p.window = window;
    santa_prefix_t x = {};
    x.n_groups = groups, x.group_offsets = p.kv_lens, x.prefix_lens = p.kv_lens;
    x.max_prefix = max_prefix, x.max_own = max_own, x.max_group = max_group;
    const santa_diff_t d = {static_cast<float*>(at), 0, nullptr, 0.f, 1.f};
    float* const s = e4m3 ? static_cast<float*>(at) : nullptr;
    const size_t bytes = 1ull << 42;
    got.clear();
    santa_status_t st;
    if (diff) st = santa_diff_attention(&p, groups ? &x : nullptr, &d, at, at, at, s, s, at, nullptr, at, bytes, nullptr);
    else if (groups) st = santa_shared_attention(&p, &x, at, at, at, s, s, at, nullptr, at, bytes, nullptr);
    else st = santa_paged_attention(&p, at, at, at, s, s, at, nullptr, at, bytes, nullptr);
    std::printf("%d%s\n", (int)st, got.c_str());
  }
  return 0;
}
