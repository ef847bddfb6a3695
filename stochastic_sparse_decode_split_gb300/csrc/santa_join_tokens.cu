// santa_join_tokens.cu -- a joined pass of few query rows per KV head: launches
// of the kernel in santa_tokens.cuh, all of whose sums go to pieces.
#include "santa_join.cuh"
#include "santa_tokens.cuh"

namespace santa {

namespace {

template <typename T, bool E4M3, int D, int R>
cudaError_t inst(const JoinArgs& a, bool behind) {
  auto kern = paged_tokens_kernel<T, E4M3, D, R, JoinArgs>;
  constexpr int smem = (int)smem_bytes<E4M3, D, R>();
  static std::atomic<unsigned long long> raised{0};
  const cudaError_t e = raise_smem((const void*)kern, smem, raised);
  if (e != cudaSuccess) return e;
  return launch_pass(kern, (unsigned)((long long)a.B * a.tiles * a.Hkv * a.splits), NT, smem, a.stream, behind, a);
}
template <typename T, bool E4M3>
cudaError_t shape(const JoinArgs& a, bool behind) {
  if (a.D == 128) return a.rows == 8 ? inst<T, E4M3, 128, 8>(a, behind) : inst<T, E4M3, 128, 16>(a, behind);
  return a.rows == 8 ? inst<T, E4M3, 64, 8>(a, behind) : inst<T, E4M3, 64, 16>(a, behind);
}

}  // namespace

cudaError_t launch_join_tokens(const JoinArgs& a, bool behind) {
  if (a.dtype == 0) return a.e4m3 ? shape<bf16_t, true>(a, behind) : shape<bf16_t, false>(a, behind);
  return a.e4m3 ? shape<fp16_t, true>(a, behind) : shape<fp16_t, false>(a, behind);
}

}  // namespace santa
