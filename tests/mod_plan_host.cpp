// The plan of a decode with modified scores (mod_plan.cuh) compiled for the host: a warp
// is 32 coroutines that take turns, a warp operation a turn of all of them.  Reads one
// problem from the arguments, plans it for every CTA and query tile, asks for the parts
// of every row as the merge does, and prints what came out for the test to check.
#include <setjmp.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
#include <ucontext.h>

#include <algorithm>
#include <functional>
#include <vector>

#include <cuda.h>
#include <cuda_runtime.h>

namespace warp {
ucontext_t back, lanes[32];
int lane;
bool over[32];
std::function<void(int)> body;
uint64_t slots[2][32];
int phase[32];

void entry(int l) {
  body(l);
  over[l] = true;
  swapcontext(&lanes[l], &back);
}
void yield() { swapcontext(&lanes[lane], &back); }
long long operations = 0, shrink_after = -1;  // a caller's mistake, after so many operations
std::function<void()> shrink;
// every lane's x, once all have given theirs
const uint64_t* exchange(uint64_t x) {
  const int l = lane, ph = phase[l];
  phase[l] ^= 1;
  slots[ph][l] = x;
  if (l == 0 && operations++ == shrink_after) shrink();
  yield();
  return slots[ph];
}
void run(std::function<void(int)> f) {
  static std::vector<char> stacks(32 << 16);
  body = f;
  for (int l = 0; l < 32; ++l) {
    over[l] = false;
    phase[l] = 0;
    getcontext(&lanes[l]);
    lanes[l].uc_stack.ss_sp = &stacks[static_cast<size_t>(l) << 16];
    lanes[l].uc_stack.ss_size = 1 << 16;
    lanes[l].uc_link = nullptr;
    makecontext(&lanes[l], reinterpret_cast<void (*)()>(entry), 1, l);
  }
  for (bool any = true; any;) {
    any = false;
    for (lane = 0; lane < 32; ++lane)
      if (!over[lane]) {
        swapcontext(&back, &lanes[lane]);
        any = true;
      }
  }
}
}  // namespace warp

template <class T>
T __shfl_sync(unsigned, T x, int from) {
  return static_cast<T>(warp::exchange(static_cast<uint64_t>(x))[from & 31]);
}
template <class T>
T __shfl_up_sync(unsigned, T x, int by) {
  const int l = warp::lane;
  return static_cast<T>(warp::exchange(static_cast<uint64_t>(x))[l >= by ? l - by : l]);
}
inline unsigned __ballot_sync(unsigned, bool x) {
  const uint64_t* all = warp::exchange(x);
  unsigned r = 0;
  for (int i = 0; i < 32; ++i) r |= static_cast<unsigned>(all[i] != 0) << i;
  return r;
}
inline unsigned __reduce_add_sync(unsigned, unsigned x) {
  const uint64_t* all = warp::exchange(x);
  uint64_t r = 0;
  for (int i = 0; i < 32; ++i) r += all[i];
  return static_cast<unsigned>(r);
}
inline int __ffs(unsigned x) { return __builtin_ffs(static_cast<int>(x)); }
inline unsigned atomicOr(unsigned* p, unsigned x) {
  const unsigned old = *p;
  *p |= x;
  return old;
}
struct Dim {
  unsigned x;
};
Dim gridDim, blockIdx;
using std::max;
using std::min;

#include "mod_plan.cuh"

using namespace attn;

int main(int argc, char** argv) {
  auto number = [&](const char* name, double otherwise) {
    const size_t n = strlen(name);
    for (int i = 1; i < argc; ++i)
      if (!strncmp(argv[i], name, n) && argv[i][n] == '=') return atof(argv[i] + n + 1);
    return otherwise;
  };
  const int B = static_cast<int>(number("B", 1)), Hkv = static_cast<int>(number("Hkv", 1));
  const int G = static_cast<int>(number("G", 1)), Np = static_cast<int>(number("Np", 0));
  const int Ncap = static_cast<int>(number("Ncap", 1));
  // lengths by a generator
  uint64_t seed = static_cast<uint64_t>(number("seed", 1)) * 2654435761u + 12345;
  const int lo = static_cast<int>(number("lo", 0)), hi = static_cast<int>(number("hi", Ncap));
  std::vector<int> lens(B);
  for (int& x : lens) {
    seed = seed * 6364136223846793005ull + 1442695040888963407ull;
    x = lo + static_cast<int>((seed >> 33) % static_cast<uint64_t>(hi - lo + 1));
  }
  warp::shrink_after = static_cast<long long>(number("shrink_after", -1));
  warp::shrink = [&] { std::fill(lens.begin(), lens.end(), 0); };

  ModKernelParams p = {};
  unsigned err = 0;
  std::vector<uint32_t> plan(B + 2, 0xABCDEF01u);
  p.err = &err;
  p.plan = plan.data();
  p.lens = lens.data();
  p.B = B;
  p.Hkv = Hkv;
  p.G = G;
  p.Hq = Hkv * G;
  p.Nk = Ncap;
  p.Np = Np;
  p.per_tile = 128 / G;
  p.row_blocks = (B + 2 * p.per_tile - 1) / (2 * p.per_tile);
  p.prefix_tiles = (Np + 127) / 128;
  p.pre_rows = B <= p.per_tile ? B * G : 256;
  p.prefix_cost = static_cast<float>(number("prefix_cost", 1.5));
  p.own_cost = static_cast<float>(number("own_cost", 1.15));
  const long long most = static_cast<long long>(Hkv) * (Np > 0 ? p.row_blocks : 0) * p.prefix_tiles +
                         static_cast<long long>(B) * Hkv * ((Ncap + 127) / 128);
  gridDim.x = static_cast<unsigned>(std::min<long long>(static_cast<long long>(number("ctas", 152)), most));

  // item: CTA, query tile, kind, KV head, first request, first tile, tiles, keys, slot
  for (blockIdx.x = 0; blockIdx.x < gridDim.x; ++blockIdx.x)
    for (int t = 0; t < 2; ++t) {
      std::vector<Work> items;
      warp::run([&](int lane) {
        Work w = {};
        plan_decode(p, t, lane, w, [&] {
          if (lane == 0) items.push_back(w);
          return true;
        });
      });
      for (const Work& w : items)
        printf("item %u %d %d %d %d %d %d %d %d\n", blockIdx.x, t, w.n < 0 ? -1 : w.kind, w.id, w.q0, w.tile0,
               w.n, w.hi, w.slot);
    }
  printf("err %u\n", err);

  CombineParams c = {};
  c.plan = plan.data();
  c.lens = lens.data();
  c.B = B;
  c.Hq = p.Hq;
  c.Hkv = Hkv;
  c.G = G;
  c.Nk = Ncap;
  c.Np = Np;
  c.row_blocks = p.row_blocks;
  c.per_tile = p.per_tile;
  c.prefix_tiles = p.prefix_tiles;
  c.pre_rows = p.pre_rows;
  c.prefix_total = prefix_total(p);
  c.ctas = gridDim.x;
  // stands for a merge whose compiler rounds the shares otherwise than the split's
  const float other = static_cast<float>(number("other", 1.0));
  auto costs = [&](auto& m) {
    if constexpr (requires { m.own_cost; }) {
      m.prefix_cost = p.prefix_cost;
      m.own_cost = p.own_cost * other;
    }
  };
  costs(c);
  // row: request, KV head, query head, first row and count of either group
  for (int b = 0; b < B; ++b)
    for (int h = 0; h < Hkv; ++h)
      for (int g = 0; g < G; g += std::max(1, G - 1)) {
        RowParts r;
        r.before(c, b, h, g);
        r.after(c, b, h, g);
        printf("row %d %d %d %lld %d %lld %d\n", b, h, g, r.first[0], r.count[0], r.first[1], r.count[1]);
      }
  printf("done %d %d %d\n", p.per_tile, p.row_blocks, p.pre_rows);
  return 0;
}
