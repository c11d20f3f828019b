"""Host-side checks of the batched tree calls (no GPU needed): layouts and refusals
before anything touches the device."""
import ctypes as C
import math
import os
import shutil
import subprocess

import pytest

from test_batch_abi import BAD_BATCH, BAD_CACHE, cache, rows

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = C.c_void_p(4096)        # never followed: each call is refused first
ODD = C.c_void_p(4100)
OFF = C.c_void_p(4098)


@pytest.fixture(scope="module")
def s():
    import substitute_speculative_decoding_gb300 as s
    return s


@pytest.fixture(scope="module")
def turn(s):
    return s.rope(64)


def test_rope_layout_matches_the_header(s, tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "sub_api.h"\nint main(void) {\n'
                   '  printf("%zu %zu %zu\\n", sizeof(sub_rope), offsetof(sub_rope, step), '
                   'offsetof(sub_rope, head_dim));\n  return 0;\n}\n')
    subprocess.run([gcc, "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o",
                    str(tmp_path / "layout")], check=True)
    out = subprocess.run([str(tmp_path / "layout")], check=True, capture_output=True, text=True)
    assert [int(x) for x in out.stdout.split()] == [C.sizeof(s.Rope), s.Rope.step.offset,
                                                    s.Rope.head_dim.offset]


def test_rope_steps_are_fractions_of_a_turn(s):
    r = s.rope(128, 5e5)
    for i in (0, 1, 40, 63):
        turns = 5e5 ** (-2 * i / 128) / (2 * math.pi)
        # a whole number of 2^-64 is at most 2^-65 off, whatever the turns
        assert abs(r.step[i] / 2.0 ** 64 - turns) <= 4 * 2.0 ** -53 * turns + 2.0 ** -65
    r = s.rope(64, freqs=[2 * math.pi * (j + 0.25) for j in range(32)])     # whole turns drop out
    assert all(abs(r.step[j] / 2.0 ** 64 - 0.25) < 1e-13 for j in range(32))
    assert list(s.rope(64, freqs=[0.0] * 32).step[:32]) == [0] * 32
    for bad in ([0.1] * 31, [0.1] * 64):
        with pytest.raises(s.SubError):
            s.rope(64, freqs=bad)
    for bad in (-1.0, float("nan"), float("inf"), 2e6):
        with pytest.raises(s.SubError):
            s.rope(64, freqs=[0.1] * 31 + [bad])
    for d, theta in ((96, 1e4), (64, 0.5), (64, float("nan")), (64, 1e13)):
        with pytest.raises(s.SubError):
            s.rope(d, theta)
    assert s._rope_init(64, 1e4, None, None) == s.SUB_EINVAL


def calls(s, turn, q8, kv, b):
    kv, b, r = C.byref(kv), C.byref(b), C.byref(turn)
    append = s._kv8_append_rope if q8 else s._kv_append_rope
    attend = s._chunk_tree_attn8 if q8 else s._chunk_tree_attn
    yield append(P, 512, 8, P, 256, P, 256, kv, 1, b, r, None, P, 512, None)
    yield attend(P, 512, 8, kv, 1, b, P, P, 2, 0.125, P, None, 0, None)


@pytest.mark.parametrize("q8", [False, True])
def test_bad_caches_and_batches_are_refused(s, turn, q8):
    for bad, word in BAD_CACHE:
        for r in calls(s, turn, q8, cache(s, q8, **bad), rows(s)):
            assert r == s.SUB_EINVAL and word in s._lib.sub_last_error(), bad
        if "n_layers" not in bad:
            move = s._kv8_move if q8 else s._kv_move
            r = move(C.byref(cache(s, q8, **bad)), 2, P, P, 3, P, None)
            assert r == s.SUB_EINVAL and word in s._lib.sub_last_error(), bad
    for bad, word in BAD_BATCH:
        for r in calls(s, turn, q8, cache(s, q8), rows(s, **bad)):
            assert r == s.SUB_EINVAL and word in s._lib.sub_last_error(), bad
    if q8:
        for name in ("k_scale", "v_scale"):
            for at, word in ((None, b"null"), (4100, b"aligned")):
                for r in calls(s, turn, True, cache(s, True, **{name: at}), rows(s)):
                    assert r == s.SUB_EINVAL and word in s._lib.sub_last_error()


def test_an_empty_batch_needs_nothing(s, turn):
    for q8 in (False, True):
        for r in calls(s, turn, q8, cache(s, q8), rows(s, n_rows=0)):
            assert r == s.SUB_OK
        move = s._kv8_move if q8 else s._kv_move
        assert move(C.byref(cache(s, q8)), 2, None, None, 0, None, None) == s.SUB_OK
    assert s._beam_select(None, None, 0, 4, 10, 1.0, 2, None, 0, -1, None, None, None, None, None, 0,
                          None) == s.SUB_OK


def test_bad_rows_are_refused(s, turn):
    kv, b, r = C.byref(cache(s)), C.byref(rows(s)), C.byref(turn)
    other = s.rope(128)

    def rope(q=P, ldq=512, hq=8, k=P, ldk=256, v=P, ldv=256, layer=0, r=r, at=None, out=P, ldo=512,
             kv=kv, b=b):
        return s._kv_append_rope(q, ldq, hq, k, ldk, v, ldv, kv, layer, b, r, at, out, ldo, None)

    def attn(q=P, ldq=512, hq=8, layer=0, base=P, mask=P, words=2, scale=0.1, out=P, ws=None, size=0):
        return s._chunk_tree_attn(q, ldq, hq, kv, layer, b, base, mask, words, scale, out, ws, size, None)

    def move(n=2, to=P, src=P, most=3, count=P, kv=kv):
        return s._kv_move(kv, n, to, src, most, count, None)
    bad = [rope(q=None), rope(out=None), rope(k=None), rope(v=None), rope(kv=None), rope(b=None),
           rope(r=None), rope(r=C.byref(other)), rope(hq=-1), rope(hq=1 << 16), rope(ldq=504),
           rope(ldq=516), rope(ldo=504, q=C.c_void_p(8192)), rope(ldk=248), rope(ldv=252), rope(q=ODD),
           rope(k=ODD), rope(out=ODD), rope(at=OFF), rope(layer=2), rope(ldq=1024), rope(ldo=1024)]
    bad += [attn(base=None), attn(mask=None), attn(words=0), attn(words=65), attn(base=OFF), attn(mask=OFF),
            attn(q=None), attn(out=None), attn(ldq=504), attn(hq=7), attn(hq=0), attn(scale=-1.0),
            attn(scale=float("nan")), attn(q=ODD), attn(ws=P, size=16), attn(ws=ODD, size=1 << 40),
            s._chunk_tree_attn(P, 512, 8, kv, 0, None, P, P, 1, 0.1, P, None, 0, None)]
    bad += [move(n=0), move(n=1025), move(to=None), move(src=None), move(count=None), move(most=-1),
            move(most=129), move(kv=None), move(to=OFF), move(src=OFF), move(count=OFF)]
    assert bad == [s.SUB_EINVAL] * len(bad)


def test_bad_beams_are_refused(s):
    place = {k: (i + 1) << 20 for i, k in enumerate(
        ("logits", "score", "state", "token", "parent", "score_out", "state_out"))}

    def call(b=2, n=3, v=10, temp=1.0, k=4, words=2, slot=-1, ws=None, size=0, **kw):
        a = {x: None if y is None else C.c_void_p(y) for x, y in {**place, **kw}.items()}
        return s._beam_select(a["logits"], a["score"], b, n, v, temp, k, a["state"], words, slot,
                              a["token"], a["parent"], a["score_out"], a["state_out"], ws, size, None)
    bad = [call(b=-1), call(b=1025), call(n=0), call(n=65), call(v=0), call(v=(1 << 20) + 1),
           call(temp=0.0), call(temp=float("nan")), call(k=0), call(k=65), call(words=0), call(slot=-2),
           call(slot=61), call(slot=2 ** 31 - 1), call(state=None), call(state_out=None),
           call(logits=None), call(score=None), call(token=None), call(parent=None), call(score_out=None),
           call(ws=P, size=16), call(ws=ODD, size=1 << 40)]
    bad += [call(**{k: v + 2}) for k, v in place.items()]
    assert bad == [s.SUB_EINVAL] * len(bad)
    size = {"logits": 60, "score": 6, "state": 12, "token": 8, "parent": 8, "score_out": 8, "state_out": 16}
    for out in ("token", "parent", "score_out", "state_out"):
        for other in size:
            if other == out:
                continue
            for x in (place[other], place[other] + 4 * (size[other] - 1), place[other] - 4 * (size[out] - 1)):
                assert call(**{out: x}) == s.SUB_EINVAL and b"apart" in s._lib.sub_last_error(), (out, other)
    n = C.c_int64()
    assert s._beam_workspace(2, 3, 10, None) == s.SUB_EINVAL
    assert s._beam_workspace(2, 0, 10, C.byref(n)) == s.SUB_EINVAL
    assert s.beam_workspace(64, 8, 152064) > 0 and s.beam_workspace(0, 8, 152064) == 0


def test_python_refuses_tensors_off_the_gpu(s):
    import torch
    with pytest.raises(s.SubError):
        s.beam_select(torch.zeros(2, 3, 4), torch.zeros(2, 3), 2)
    with pytest.raises(s.SubError):
        s.kv_move(cache(s), torch.zeros(1, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32),
                  torch.zeros(1, dtype=torch.int32))
