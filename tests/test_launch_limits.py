"""CPU: the launches of the largest calls that the cache and adapter entry points accept. A recorder in
place of the HIP runtime's launch takes down each launch's grid, so nothing runs and no pointer is followed. HIP
has 32 bits for the threads of a grid's dimension."""
import json
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
RECORDER = r"""
#include <stdint.h>
#include <stddef.h>
typedef struct { uint32_t x, y, z; } dim3;
static uint32_t log_[64][6];
static int count_;
int hipLaunchKernel(const void* f, dim3 g, dim3 b, void** args, size_t lds, void* stream) {
  (void)f; (void)args; (void)lds; (void)stream;
  if (count_ < 64) {
    uint32_t* o = log_[count_++];
    o[0] = g.x; o[1] = g.y; o[2] = g.z; o[3] = b.x; o[4] = b.y; o[5] = b.z;
  }
  return 0;
}
int hipGetLastError(void) { return 0; }
/* what <<< >>> hands to the launch; the runtime's own needs a device */
static dim3 grid_, block_;
int __hipPushCallConfiguration(dim3 g, dim3 b, size_t lds, void* stream) {
  (void)lds; (void)stream;
  grid_ = g; block_ = b;
  return 0;
}
int __hipPopCallConfiguration(dim3* g, dim3* b, size_t* lds, void** stream) {
  *g = grid_; *b = block_; *lds = 0; *stream = 0;
  return 0;
}
int launches_taken(uint32_t* out) {
  const int n = count_;
  for (int i = 0; i < n; ++i) for (int j = 0; j < 6; ++j) out[6 * i + j] = log_[i][j];
  count_ = 0;
  return n;
}
"""

PROGRAM = r"""
import ctypes, json, sys
rec = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)  # before the HIP runtime
sys.path.insert(0, sys.argv[2])
from mxfp4_block_scaled_hadamard32_amd import _lib as m
L, P = m.lib(), lambda i: i << 52
rows = lambda i, heads, dim: ctypes.byref(m.mx_rows(P(i), heads * dim, dim))

def cache(offsets=True, **kw):
    v = dict(kq=P(1), ks=P(2), vq=P(3), vs=P(4), pages=P(5), lengths=P(6),
             offsets=P(7) if offsets else None, n_pages=1000, seqs=64, table_width=256, heads=8,
             dim=64, page_size=64, fmt=0)
    v.update(kw)
    return ctypes.byref(m.mx_cache(**v))

def attention(T, q_heads, **kw):
    c = cache(**kw)
    dim = kw.get("dim", 64)
    size = L.mx_cache_attention_workspace(T, q_heads, c)
    return L.mx_cache_attention(rows(8, q_heads, dim), rows(9, q_heads, dim), P(10), 1, T, q_heads, 0.1, c,
                                P(11), size, None)

def write(T, **kw):
    h, d = kw.get("heads", 8), kw.get("dim", 64)
    return L.mx_cache_write(rows(8, h, d), rows(9, h, d), 1, T, cache(**kw), 0, None)

def read(T, **kw):
    h, d = kw.get("heads", 8), kw.get("dim", 64)
    return L.mx_cache_read(rows(8, h, d), rows(9, h, d), 1, T, cache(**kw), None)

def lora(T, N, K, E, r, dtype):
    size = L.mx_lora_workspace(dtype, T, N, K, E, r)
    return L.mx_lora(P(1), dtype, K, P(2), P(3), E, r, P(4), P(5), P(6), 0, N, T, N, K, dtype, P(7), N, P(8),
                     size, None)

out = []
for name, args, kw in json.loads(sys.argv[3]):
    status = {"attention": attention, "write": write, "read": read, "lora": lora}[name](*args, **kw)
    taken = (ctypes.c_uint32 * 384)()
    n = rec.launches_taken(taken)
    out.append([status, [list(taken[6 * i:6 * i + 6]) for i in range(n)]])
print(json.dumps(out))
"""

M = 1 << 20
CALLS = [  # and how many launches
    ("attention", [M, 64], {}, 2),                                 # 2^26 rows, prompts of 16384 tokens
    ("attention", [M, 63], {"heads": 7}, 2),
    ("attention", [16 * M, 64], {"heads": 64, "table_width": 8}, 2),  # 2^30 rows
    ("attention", [16 * M, 64], {"heads": 1, "table_width": 8, "seqs": 1}, 2),
    ("attention", [M, 1024], {"offsets": False, "seqs": M, "heads": 1024, "table_width": 2, "dim": 256}, 2),
    ("attention", [16 * M, 64], {"heads": 64, "table_width": 1}, 1),
    ("attention", [2048, 65535], {"heads": 65535, "table_width": 8}, 2),
    ("attention", [1, 1], {"heads": 1, "seqs": 1, "table_width": 16}, 1),
    ("attention", [1, 2047], {"heads": 1, "seqs": 1}, 2), ("attention", [1, 2048], {"heads": 1, "seqs": 1}, 2),
    ("write", [16 * M], {"seqs": M, "dim": 256, "heads": 65535}, 1),
    ("read", [16 * M], {"seqs": M, "dim": 256, "heads": 65535}, 1),
    ("write", [M], {"offsets": False, "seqs": M, "dim": 256}, 1),
    ("lora", [2 * M, 64 * M, 4096, 1024, 128, 0], {}, 2), ("lora", [2 * M, 64 * M, 64 * M, 64, 128, 1], {}, 2),
    ("lora", [16, 16384, 4096, 16, 16, 1], {}, 1), ("lora", [1, 64 * M, 4096, 1, 16, 1], {}, 2),
]


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    from mxfp4_block_scaled_hadamard32_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("libmx.so not built (run __graft_entry__.build())")
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    d = tmp_path_factory.mktemp("recorder")
    (d / "recorder.c").write_text(RECORDER)
    lib = str(d / "recorder.so")
    subprocess.run([cc, "-O1", "-shared", "-fPIC", "-Wall", "-Wextra", "-Werror", "-o", lib,
                    str(d / "recorder.c")], check=True)
    res = subprocess.run([sys.executable, "-c", PROGRAM, lib, ROOT, json.dumps([c[:3] for c in CALLS])],
                         capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr
    return json.loads(res.stdout.splitlines()[-1])


@pytest.mark.parametrize("i", range(len(CALLS)), ids=lambda i: f"{CALLS[i][0]}-{i}")
def test_grids(launches, i):
    status, taken = launches[i]
    assert status == 0 and len(taken) == CALLS[i][3], (status, taken)
    for gx, gy, gz, bx, by, bz in taken:
        assert min(gx, gy, gz) >= 1 and bx * by * bz <= 1024
        assert gx * bx < 1 << 32 and gy * by < 1 << 32 and gz * bz < 1 << 32, (gx, gy, gz, bx)
        assert gy <= 65535 and gz <= 65535, (gx, gy, gz)


def test_every_row_is_joined(launches):
    """The second launch of the attention has a thread group for each row: a workgroup below 2048
    rows, a wave from there on."""
    for (name, args, kw, count), (_, taken) in zip(CALLS, launches):
        if name == "attention" and count == 2:
            rows = args[0] * args[1]
            gx, gy, gz, bx, _, _ = taken[1]
            assert gx * gy * gz * (bx // (256 if rows < 2048 else 64)) >= rows
