"""GPU test: a process whose first decode calls, 8-bit and 16-bit, come from several host threads at
the same moment, with groups of one kernel variant that need different amounts of shared memory.
Every call is launched, then and later."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

# n threads that meet at a spinning barrier and make one call each
AT_ONCE = r"""
#include <atomic>
#include <thread>
#include <vector>
#include "pa.h"
struct Arg { int group; float *out; void *q, *workspace; pa_stream_t stream; };
struct Pool { void *codes, *pool; float *scale; int32_t *table, *lens; size_t workspace_bytes; int blocks; };
extern "C" void at_once(decltype(&pa_paged_decode_attention_fp8) eight, decltype(&pa_paged_decode_attention) sixteen,
                        decltype(&pa_device_error) error, int n, const Arg *a, const Pool *p, int *status) {
  std::atomic<int> here{0};
  std::vector<std::thread> threads;
  for (int i = 0; i < n; ++i)
    threads.emplace_back([=, &here] {
      unsigned flags;
      error(&flags, 0);                     // the thread has a context
      ++here;
      while (here.load() < n) {}
      const Arg &x = a[i];
      const int len = p->blocks * 16;
      status[i] = eight ? eight(x.out, x.q, p->codes, p->codes, p->scale, p->table, p->lens, 1.f, 1, 1, x.group,
                                128, 16, p->blocks, len, p->blocks, PA_F16, x.workspace, p->workspace_bytes, x.stream)
                        : sixteen(x.out, x.q, p->pool, p->pool, p->table, p->lens, 1.f, 1, 1, x.group, 128, 16,
                                  p->blocks, len, p->blocks, PA_F16, x.workspace, p->workspace_bytes, x.stream);
    });
  for (auto &t : threads) t.join();
}
"""

FIRST_CALLS = """
import ctypes as c, sys
import torch
import paged_kv_cache_414_b200 as pa
helper, eight = c.CDLL(sys.argv[1]), sys.argv[2] == "8"
L, D, B, NB = pa.lib(), 128, 16, 8
Arg = type("Arg", (c.Structure,), {"_fields_": [("group", c.c_int)] + [(x, c.c_void_p) for x in (
    "out", "q", "workspace", "stream")]})
Pool = type("Pool", (c.Structure,), {"_fields_": [(x, c.c_void_p) for x in (
    "codes", "pool", "scale", "table", "lens")] + [("bytes", c.c_size_t), ("blocks", c.c_int)]})
pool = torch.zeros(NB, 1, B, D, dtype=torch.float16, device="cuda")
codes, scale = pool.to(torch.float8_e4m3fn), torch.ones(NB, 1, 2, B, device="cuda")
table, lens = torch.arange(NB, device="cuda").int(), torch.full((1,), NB * B, dtype=torch.int32, device="cuda")
groups = [16, 9, 16, 9]
outs = [torch.ones(1, G, D, device="cuda") for G in groups]
qs = [torch.zeros(1, G, D, dtype=torch.float16, device="cuda") for G in groups]
spaces = [pa.alloc_workspace(1, 16, 1, D, B, NB * B) for _ in groups]
streams = [torch.cuda.Stream() for _ in groups]
args = (Arg * len(groups))(*[Arg(G, o.data_ptr(), q.data_ptr(), w.data_ptr(), s.cuda_stream)
                             for G, o, q, w, s in zip(groups, outs, qs, spaces, streams)])
p = Pool(codes.data_ptr(), pool.data_ptr(), scale.data_ptr(), table.data_ptr(), lens.data_ptr(),
         spaces[0].numel(), NB)
torch.cuda.synchronize()
address = lambda f: c.cast(f, c.c_void_p)
seen = []
for _ in range(2):
    status = (c.c_int * len(groups))()
    helper.at_once(address(L.pa_paged_decode_attention_fp8) if eight else None,
                   address(L.pa_paged_decode_attention), address(L.pa_device_error), len(groups), args,
                   c.byref(p), status)
    seen += list(status)
torch.cuda.synchronize()
assert seen == [0] * len(seen), seen
assert all((o == 0).all() for o in outs) and pa.pa_device_error() == 0
"""


@pytest.mark.parametrize("bits", [8, 16])
def test_first_calls_at_the_same_moment(pa, cuda_device, tmp_path, bits):
    root = os.path.dirname(os.path.dirname(os.path.abspath(pa.__file__)))
    source, helper = tmp_path / "at_once.cpp", tmp_path / "at_once.so"
    source.write_text(AT_ONCE)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-pthread", "-I", os.path.join(root, "include"),
                    str(source), "-o", str(helper)], check=True)
    for _ in range(2):
        r = subprocess.run([sys.executable, "-c", FIRST_CALLS, str(helper), str(bits)], cwd=root,
                           capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stderr[-2000:]
