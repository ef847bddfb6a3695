// santa_join_tokens.cu -- joined passes of few query rows per KV head: the work of
// santa_tokens.cuh, all of whose sums go to pieces.
//
// Where both passes are of few rows one launch has both, the prefixes' CTAs
// first: four tokens behind 600 keys 9.0 -> 8.3 us, called from Python among
// others 12.3 -> 10.3.
#include "santa_join.cuh"
#include "santa_tokens.cuh"

namespace santa {

namespace {

template <typename T, bool E4M3, int D, int R>
__global__ void __launch_bounds__(NT, E4M3 ? 3 : 2) join_tokens_kernel(const __grid_constant__ JoinArgs a) {
  paged_tokens<T, E4M3, D, R>(a, blockIdx.x, blockIdx.x == 0);
}
template <typename T, bool E4M3, int D, int R0, int R1>
__global__ void __launch_bounds__(NT, E4M3 ? 3 : 2) both_tokens_kernel(const __grid_constant__ Passes p, unsigned first) {
  if (blockIdx.x < first) paged_tokens<T, E4M3, D, R0>(p.p[0], blockIdx.x, false);
  else paged_tokens<T, E4M3, D, R1>(p.p[1], blockIdx.x - first, false);
}

template <typename T, bool E4M3, int D, int R0, int R1>
cudaError_t both(const JoinArgs& p, const JoinArgs& a) {
  constexpr int s0 = (int)smem_bytes<E4M3, D, R0>(), s1 = (int)smem_bytes<E4M3, D, R1>(), smem = s0 > s1 ? s0 : s1;
  auto kern = both_tokens_kernel<T, E4M3, D, R0, R1>;
  static std::atomic<unsigned long long> raised{0};
  const cudaError_t e = raise_smem((const void*)kern, smem, raised);
  if (e != cudaSuccess) return e;
  const unsigned first = (unsigned)tokens_grid(p);
  return launch_pass(kern, first + (unsigned)tokens_grid(a), NT, smem, a.stream, false, Passes{{p, a}}, first);
}
template <typename T, bool E4M3, int D, int R>
cudaError_t one(const JoinArgs& a, bool behind) {
  constexpr int smem = (int)smem_bytes<E4M3, D, R>();
  auto kern = join_tokens_kernel<T, E4M3, D, R>;
  static std::atomic<unsigned long long> raised{0};
  const cudaError_t e = raise_smem((const void*)kern, smem, raised);
  if (e != cudaSuccess) return e;
  return launch_pass(kern, (unsigned)tokens_grid(a), NT, smem, a.stream, behind, a);
}
template <typename T, bool E4M3, int D>
cudaError_t rows(const JoinArgs* p, const JoinArgs& a, bool behind) {
  if (!p) return a.rows == 8 ? one<T, E4M3, D, 8>(a, behind) : one<T, E4M3, D, 16>(a, behind);
  if (p->rows == 8) return both<T, E4M3, D, 8, 8>(*p, a);   // a sequence has no more rows than its group
  return a.rows == 8 ? both<T, E4M3, D, 16, 8>(*p, a) : both<T, E4M3, D, 16, 16>(*p, a);
}
template <typename T>
cudaError_t type(const JoinArgs* p, const JoinArgs& a, bool behind) {
  if (a.D == 128) return a.e4m3 ? rows<T, true, 128>(p, a, behind) : rows<T, false, 128>(p, a, behind);
  return a.e4m3 ? rows<T, true, 64>(p, a, behind) : rows<T, false, 64>(p, a, behind);
}

}  // namespace

cudaError_t launch_join_tokens(const JoinArgs* prefixes, const JoinArgs& a, bool behind) {
  return a.dtype == 0 ? type<bf16_t>(prefixes, a, behind) : type<fp16_t>(prefixes, a, behind);
}

}  // namespace santa
