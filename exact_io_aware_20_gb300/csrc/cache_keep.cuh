// The window of a sequence whose last tokens are thinned (fa_cache_pages.cu).
#pragma once

namespace fa {

struct KeepWindow {
  int base, end;      // the first token of the window, and behind the last kept one's place
  bool valid;         // otherwise nothing of the sequence is read or moved
};

// Of the last n of `len` tokens `kept` stay; N and K are the most that there may
// be of either, `capacity` the tokens that a row of the block table has pages for.
// More kept tokens than there are in the window cannot have numbers that rise and
// stay below n: refused here, ahead of the first read of the row, which they would
// leave where the window ends at its last page.
__host__ __device__ __forceinline__ KeepWindow keep_window(int len, int n, int kept, int N, int K, long long capacity) {
  const bool valid = n >= 0 && n <= N && len >= n && len <= capacity && kept >= 0 && kept <= K &&
                     kept <= n;
  const int base = valid ? len - n : 0;
  return {base, base + (valid ? kept : 0), valid};
}

}  // namespace fa
