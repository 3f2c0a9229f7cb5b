"""What the header promises of the speculative step's host side, at its edges (CPU)."""
import math
import os
import shutil
import subprocess

import numpy as np
import pytest

import non_uniform_paged_flash_b200 as tg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _plan(cap, T=4, Hq=8, Hkv=2, D=128, pages=1 << 20, workers=0):
    B = np.asarray(cap).size // Hkv
    return tg.tg_tree_plan_create(tg.make_shape(B, Hq, Hkv, D, pages), cap, T, np.zeros(Hkv, np.int32), [0, 1 << 20],
                                  num_workers=workers, host_only=True)


@pytest.mark.parametrize("cap,ok", [([0, 0], True), ([0, 1], False), ([40, 0], False)])
def test_plan_needs_a_pool_for_reserved_tokens(cap, ok):
    """Heads that reserve tokens need pages to hold them: with an empty pool there is no page a bad
    page id could be replaced by."""
    if ok:
        assert tg.tg_tree_plan_items(_plan(cap, pages=0))["n_items"] == 2
        return
    with pytest.raises(tg.TGError) as e:
        _plan(cap, pages=0)
    assert e.value.status == tg.TG_EINVAL


@pytest.mark.parametrize("T,G", [(16, 4), (4, 4), (64, 8)])
@pytest.mark.parametrize("full,tokens", [(0, 0), (1, 600), (16, 64), (8, 1000), (60, 100), (300, 17), (256, 4000)])
def test_plan_spreads_heads_without_tokens(T, G, full, tokens):
    """A head that reserves nothing still has its drafted tokens: such heads are dealt out with the rest."""
    BH = 512
    cap = np.zeros(BH, np.int32)
    cap[np.random.default_rng(0).permutation(BH)[:full]] = tokens
    info = tg.tg_tree_plan_items(_plan(cap, T=T, Hq=8 * G, Hkv=8))
    it, off = info["items"], info["worker_off"]
    # an even share of the (head, row block) units, and as many more as a worker's share of the pages
    # amounts to: a page is worth a unit at most in a step bound by latency, 1/18 of one in others
    units, workers = BH * (2 if T * G > 256 else 1), info["n_workers"]
    pages = units * full * -(-tokens // 16) / BH
    per = np.diff(off)
    assert per.max() <= units / workers + max(4, pages / (18 * workers)) + 2
    if pages < 4 * workers:
        assert off[-1] == len(it)                             # none by ticket
        load = [int(np.maximum(it[a:b, 2] - it[a:b, 1], 1).sum()) for a, b in zip(off[:-1], off[1:])]
        assert max(load) <= (pages + units) / workers + 12


def test_default_stream_before_cuda_is_up(monkeypatch):
    """Without a stream argument a call asks torch for its current stream, which brings CUDA up or says why it
    cannot be (no CUDA build, a forked child), with or without the entries that are faster once it is up."""
    import torch

    class Stream:
        cuda_stream = 77

    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream)
    assert tg._stream(None) == 77
    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name, raising=False)
    assert tg._stream(None) == 77
    assert tg._stream(5) == 5 and tg._stream(Stream) == 77

    def no_cuda():
        raise AssertionError("Torch not compiled with CUDA enabled")

    monkeypatch.setattr(torch.cuda, "current_stream", no_cuda)
    with pytest.raises(AssertionError):
        tg._stream(None)


@pytest.mark.parametrize("orig,fast,slow", [(4096, 32.0, 1.0), (5, 32.0, 1.0), (1, 2.0, 0.5), (100, 50.0, 20.0),
                                             (1 << 40, 32.0, 1.0), (64, 10.18, 10.0), (7, 1.2, 1.1)])
@pytest.mark.parametrize("rot,base", [(64, 10000.0), (2, 10000.0), (128, 1.5), (10, 5e5)])
def test_yarn_keeps_fast_pairs_and_interpolates_slow_ones(rot, base, orig, fast, slow):
    """By the turns of each pair over the original length, also where every pair is slow or every one fast."""
    plain = tg.tg_rope_frequencies(rot, base)[0]
    yarn = tg.tg_rope_frequencies(rot, base, tg.TG_ROPE_YARN, 8.0, orig, fast, slow)[0]
    turns = orig * plain / (2 * math.pi)
    np.testing.assert_allclose(yarn[turns > fast], plain[turns > fast], rtol=1e-12)
    np.testing.assert_allclose(yarn[turns < slow], plain[turns < slow] / 8, rtol=1e-12)
    assert np.all(yarn <= plain * (1 + 1e-12)) and np.all(yarn >= plain / 8 * (1 - 1e-12))


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_masks_refuse_offsets_out_of_order_unread(tmp_path):
    exe, csrc = str(tmp_path / "mask_bounds"), os.path.join(ROOT, "non_uniform_paged_flash_b200", "csrc")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                           "-I" + os.path.join(ROOT, "include"), "-I" + csrc,
                           os.path.join(ROOT, "tests", "native", "mask_bounds.cpp"),
                           os.path.join(csrc, "tg_host.cpp"), "-o", exe])
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "refused" in r.stdout
