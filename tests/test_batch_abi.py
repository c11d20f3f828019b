"""Host-side checks of the batched calls (no GPU needed): struct layouts, and
refusals before anything touches the device."""
import ctypes as C
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = C.c_void_p(4096)        # never followed: each call is refused first
ODD = C.c_void_p(4100)


@pytest.fixture(scope="module")
def s():
    import substitute_speculative_decoding_gb300 as s
    return s


def test_struct_layouts_match_the_header(s, tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    mirrors = {"sub_batch": s.Batch, "sub_kv8_cache": s.KV8Cache}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "sub_api.h"', "int main(void) {"]
    for c, py in mirrors.items():
        lines.append(f'  printf("%zu\\n", sizeof({c}));')
        lines += [f'  printf("%zu\\n", offsetof({c}, {f[0]}));' for f in py._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    subprocess.run([gcc, "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o",
                    str(tmp_path / "layout")], check=True)
    out = subprocess.run([str(tmp_path / "layout")], check=True, capture_output=True, text=True)
    want = []
    for py in mirrors.values():
        want.append(C.sizeof(py))
        want += [getattr(py, f[0]).offset for f in py._fields_]
    assert [int(x) for x in out.stdout.split()] == want


def cache(s, q8=False, **kw):
    kv = (s.KV8Cache if q8 else s.KVCache)()
    kv.k = kv.v = kv.page_table = 4096
    if q8:
        kv.k_scale = kv.v_scale = 4096
    kv.n_layers, kv.n_heads_kv, kv.head_dim, kv.page_size, kv.n_pages = 2, 4, 64, 16, 8
    kv.capacity = 64
    for k, v in kw.items():
        setattr(kv, k, v)
    return kv


def rows(s, **kw):
    b = s.Batch(4096, 4096, 2, 5, 0)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


BAD_CACHE = [({"head_dim": 96}, b"head_dim"), ({"page_size": 24}, b"page_size"),
             ({"page_size": 0}, b"page_size"), ({"n_pages": 0}, b"cache sizes"),
             ({"capacity": 0}, b"cache sizes"), ({"capacity": 1 << 31}, b"cache sizes"),
             ({"n_heads_kv": 0}, b"n_heads_kv"), ({"k": None}, b"null"), ({"v": 4100}, b"aligned"),
             ({"page_table": None}, b"null"), ({"n_layers": 1}, b"layer")]
BAD_BATCH = [({"start": None}, b"null"), ({"pos": None}, b"null"), ({"n_seqs": 0}, b"n_seqs"),
             ({"n_seqs": 1025}, b"n_seqs"), ({"n_rows": -1}, b"n_rows"),
             ({"n_rows": 1 << 25}, b"n_rows"), ({"max_keys": -1}, b"max_keys")]


def calls(s, q8, kv, b):
    kv, b = C.byref(kv), C.byref(b)
    if q8:
        yield s._kv8_append(P, 256, P, 256, kv, 1, b, None)
        yield s._kv8_read(kv, 1, b, P, P, None)
        yield s._chunk_attn8(P, 512, 8, kv, 1, b, 0.125, P, None, 0, None)
    else:
        yield s._kv_append(P, 256, P, 256, kv, 1, b, None)
        yield s._chunk_attn(P, 512, 8, kv, 1, b, 0.125, P, None, 0, None)


@pytest.mark.parametrize("q8", [False, True])
def test_bad_caches_and_batches_are_refused(s, q8):
    for bad, word in BAD_CACHE:
        for r in calls(s, q8, cache(s, q8, **bad), rows(s)):
            assert r == s.SUB_EINVAL and word in s._lib.sub_last_error(), bad
    for bad, word in BAD_BATCH:
        for r in calls(s, q8, cache(s, q8), rows(s, **bad)):
            assert r == s.SUB_EINVAL and word in s._lib.sub_last_error(), bad
    if q8:
        for name in ("k_scale", "v_scale"):
            for at, word in ((None, b"null"), (4100, b"aligned")):
                for r in calls(s, True, cache(s, True, **{name: at}), rows(s)):
                    assert r == s.SUB_EINVAL and word in s._lib.sub_last_error()


def test_an_empty_batch_needs_nothing(s):
    for q8 in (False, True):
        for r in calls(s, q8, cache(s, q8), rows(s, n_rows=0)):
            assert r == s.SUB_OK
    assert s._probs(None, 0, 10, 1.0, None, None) == s.SUB_OK
    assert s._verify_sample(None, None, None, None, 0, 3, 10, None, None, None) == s.SUB_OK


def test_bad_rows_are_refused(s):
    kv, k8, b = C.byref(cache(s)), C.byref(cache(s, True)), C.byref(rows(s))
    bad = [s._kv_append(None, 256, P, 256, kv, 0, b, None),
           s._kv_append(P, 255, P, 256, kv, 0, b, None),
           s._kv_append(P, 256, P, 248, kv, 0, b, None),
           s._kv_append(P, 256, ODD, 256, kv, 0, b, None),
           s._kv_append(P, 256, P, 256, kv, -1, b, None),
           s._kv_append(P, 256, P, 256, None, 0, b, None),
           s._kv_append(P, 256, P, 256, kv, 0, None, None),
           s._kv8_read(k8, 0, b, P, None, None),
           s._kv8_read(k8, 0, b, ODD, P, None),
           s._chunk_attn(None, 512, 8, kv, 0, b, 0.1, P, None, 0, None),
           s._chunk_attn(P, 512, 8, kv, 0, b, 0.1, None, None, 0, None),
           s._chunk_attn(P, 504, 8, kv, 0, b, 0.1, P, None, 0, None),
           s._chunk_attn(P, 512, 7, kv, 0, b, 0.1, P, None, 0, None),
           s._chunk_attn(P, 512, 0, kv, 0, b, 0.1, P, None, 0, None),
           s._chunk_attn(P, 1 << 16, 65 * 4, kv, 0, b, 0.1, P, None, 0, None),
           s._chunk_attn(P, 512, 8, kv, 0, b, float("nan"), P, None, 0, None),
           s._chunk_attn(P, 512, 8, kv, 0, b, -1.0, P, None, 0, None),
           s._chunk_attn(ODD, 512, 8, kv, 0, b, 0.1, P, None, 0, None),
           s._chunk_attn(P, 512, 8, kv, 0, b, 0.1, P, P, 16, None),
           s._chunk_attn(P, 512, 8, kv, 0, b, 0.1, P, ODD, 1 << 40, None),
           s._chunk_attn_workspace(8, 4, 64, 2, 5, None)]
    n = C.c_int64()
    bad += [s._chunk_attn_workspace(8, 3, 64, 2, 5, C.byref(n)),
            s._chunk_attn_workspace(8, 4, 80, 2, 5, C.byref(n)),
            s._chunk_attn_workspace(8, 4, 64, 0, 5, C.byref(n))]
    assert bad == [s.SUB_EINVAL] * len(bad)


def test_bad_probabilities_are_refused(s):
    bad = [s._probs(P, 1, 0, 1.0, P, None), s._probs(P, 1, (1 << 20) + 1, 1.0, P, None),
           s._probs(P, -1, 10, 1.0, P, None), s._probs(P, 1, 10, 0.0, P, None),
           s._probs(P, 1, 10, float("nan"), P, None), s._probs(P, 1, 10, float("inf"), P, None),
           s._probs(None, 1, 10, 1.0, P, None), s._probs(P, 1, 10, 1.0, ODD, None)]

    def ver(p=P, q=P, draft=P, u=P, n=1, k=2, v=10, tokens=P, acc=P):
        return s._verify_sample(p, q, draft, u, n, k, v, tokens, acc, None)
    bad += [ver(p=None), ver(draft=None), ver(u=None), ver(tokens=None), ver(acc=None), ver(n=-1),
            ver(k=-1), ver(v=0), ver(v=(1 << 20) + 1), ver(p=ODD), ver(q=ODD)]
    assert bad == [s.SUB_EINVAL] * len(bad)


def test_python_refuses_tensors_off_the_gpu(s):
    import torch
    with pytest.raises(s.SubError):
        s.probs(torch.zeros(2, 4))
    with pytest.raises(s.SubError):
        s.batch(torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 4)
    with pytest.raises(s.SubError):
        z = torch.zeros(1, 2, 1, 16, 64, dtype=torch.bfloat16)
        s.paged_kv(z, z, torch.zeros(1, 2, dtype=torch.int32))
