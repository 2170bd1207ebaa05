"""The 16-bit cache's calls together, as an engine runs them, and next to the codec and the 8-bit cache."""
import importlib.util
import os

import pytest
import torch

import cache8_ref as R8
import cache16_ref as R
from kv_cache_page_gb300 import cache8, cache16
from test_gpu_cache16 import _check

pytestmark = pytest.mark.gpu
DEV = "cuda"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("serve_cache16", os.path.join(ROOT, "examples", "serve_cache16.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_the_example_serves_offloads_and_goes_on():
    """examples/serve_cache16.py end to end, small: the last step's outputs are the attention over the pages as they
    lie then, restored ones among them, of the queries as they were turned."""
    r = _example().serve(3, 90, 20)
    assert not r["errors"].any() and r["restored"] == r["segments"] == 2 * 7
    lens = [90 + 22, 73 + 22, 56 + 22]
    assert r["lens"].tolist() == lens
    su = R.Setup(D=128, H=8, T=16, lens=lens, dtype="bf16")
    pages = r["pages"].cpu().transpose(1, 2)
    su.pool, su.tables, su.pages = [pages[..., :128], pages[..., 128:]], r["tables"].cpu(), pages.shape[0]
    _check(su, lens, None, r["step_q"].cpu(), r["step_out"].cpu().double(), r["step_lse"].cpu().double())
    for name in ("out", "draft_out"):
        assert torch.isfinite(r[name].float()).all()
    # the prompts' queries, turned by the positions of their rows
    pos = [p for n in (90, 73, 56) for p in range(n)]
    tab = r["rotation"].cos.cpu(), r["rotation"].sin.cpu()
    assert torch.equal(R.turn(r["prompt_q"].cpu().float(), pos, *tab, False).to(torch.bfloat16), r["prompt_turned"].cpu())


def test_the_example_s_prompts_and_drafts(monkeypatch):
    """What the example's calls outside its graph give, the prompts' and the drafts', is the attention over the pages as
    they lie at that time."""
    calls, attend = [], cache16.Cache16.attend

    def kept(self, layer, batch, q, out, **kw):
        attend(self, layer, batch, q, out, **kw)
        if not torch.cuda.is_current_stream_capturing():
            calls.append([x.cpu() for x in (batch.tables, batch.lens, batch.cu_new, q, out, layer.k, layer.v)])

    monkeypatch.setattr(cache16.Cache16, "attend", kept)
    _example().serve(3, 90, 20)
    assert [c[3].shape[0] for c in calls] == [90 + 73 + 56, 3 * 4]
    for tables, lens, cu, q, out, k, v in calls:
        su = R.Setup(D=128, H=8, T=16, lens=lens.tolist(), dtype="bf16")
        su.pool, su.tables, su.pages = [k.transpose(1, 2), v.transpose(1, 2)], tables, k.shape[0]
        for s in range(3):
            rows = slice(int(cu[s]), int(cu[s + 1]))
            want, _, eo, _ = su.attend(s, int(lens[s]), q[rows])
            assert bool(((out[rows].double() - want).abs() <= eo).all()), s


def test_one_batch_serves_16_bit_and_8_bit_layers():
    """A model with layers of both kinds: one batch, one rotation and one workspace; prompts, then single tokens."""
    lens = [70, 33, 5]
    s16 = R.Setup(D=64, H=2, T=16, lens=[n + 3 for n in lens], dtype="bf16", seed=1)
    s8 = R8.Setup(D=64, H=2, T=16, lens=[n + 3 for n in lens], dtype="bf16", seed=1)
    s8.tables, s8.pages = s16.tables.clone(), s16.pages
    s8.ref = R8.Cache(s8.pages, 16, 2, 64)
    c16, c8 = s16.cache(cache16, 4), s8.cache(cache8, 4)
    y16, y8 = s16.device_layer(cache16), s8.device_layer(cache8)
    cos, sin = R.tables(100, 32)
    rotation = cache8.Rotation(cos.to(DEV), sin.to(DEV), interleaved=True)
    ws = None
    for step in range(4):
        new = lens if step == 0 else None
        now = [n + step for n in lens]
        b = s16.batch(cache8, new, now)
        if ws is None:
            ws = torch.zeros(max(c16.attend_workspace(b), c8.attend_workspace(b)), dtype=torch.uint8, device=DEV)
        rows = [(s, now[s] - c + i) for s, c in enumerate(new or [1] * 3) for i in range(c)]
        n = len(rows)
        k, v, q = s16.values(n), s16.values(n), s16.values(n, 4)
        turned = R.turn(k.float(), [p for _, p in rows], cos, sin, True)
        outs = []
        for c, y in ((c16, y16), (c8, y8)):
            qo, out, lse = torch.empty(n, 4, 64, dtype=s16.dtype, device=DEV), torch.empty(n, 4, 64, dtype=s16.dtype, device=DEV), \
                torch.empty(n, 4, device=DEV)
            c.append(y, b, k.to(DEV), v.to(DEV), rotation=rotation, q=q.to(DEV), q_out=qo)
            c.attend(y, b, qo, out, lse=lse, workspace=ws)
            outs.append((qo.cpu(), out.cpu().double(), lse.cpu().double()))
        assert torch.equal(outs[0][0], outs[1][0])
        at = 0
        for s, c in enumerate(new or [1] * 3):
            s16.put(s, now[s] - c, turned[at:at + c].to(s16.dtype), v[at:at + c])
            s8.ref.write(s8.tables[s], now[s] - c, (turned[at:at + c], v[at:at + c]))
            at += c
        _check(s16, now, new, *outs[0])
        from test_gpu_cache8 import _check as check8
        check8(s8, now, new, *outs[1])


def test_two_streams_with_workspaces_of_their_own():
    """Calls that may run at the same time, each with its own workspace, give what they give alone."""
    lens = [6000, 40, 900]
    su = R.Setup(D=128, H=2, T=16, lens=lens, dtype="fp16", seed=6)
    su.fill()
    c, layer, b = su.cache(cache16, 8), su.device_layer(cache16), su.batch(cache8)
    q = su.values(3, 8).to(DEV)
    size = c.attend_workspace(b)
    want = torch.empty_like(q)
    c.attend(layer, b, q, want, workspace=torch.zeros(size, dtype=torch.uint8, device=DEV))
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [torch.zeros(size, dtype=torch.uint8, device=DEV) for _ in range(2)]
    outs = [[torch.empty_like(q) for _ in range(8)] for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(8):
        for s in range(2):
            c.attend(layer, b, q, outs[s][i], workspace=spaces[s], stream=streams[s])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for s in outs for o in s)


def test_two_captured_graphs_share_a_workspace_in_turn():
    lens = [5000, 40, 900]
    su = R.Setup(D=64, H=2, T=16, lens=lens, dtype="fp16", seed=6)
    su.fill()
    c, layer = su.cache(cache16, 8), su.device_layer(cache16)
    batches = [su.batch(cache8), su.batch(cache8, [3, 1, 2])]
    qs = [su.values(n, 8).to(DEV) for n in (3, 6)]
    size = c.attend_workspace(batches[0])
    shared, graphs, outs, wants = torch.zeros(size, dtype=torch.uint8, device=DEV), [], [], []
    for b, q in zip(batches, qs):
        want, out = torch.empty_like(q), torch.empty_like(q)
        c.attend(layer, b, q, want, workspace=torch.zeros(size, dtype=torch.uint8, device=DEV))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.attend(layer, b, q, out, workspace=shared)
        graphs.append(g), outs.append(out), wants.append(want)
    for i in (0, 1, 1, 0, 0, 1, 0):
        outs[i].zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], wants[i]), i


def test_debug_library_sees_no_access_outside_the_buffers():
    """Append and attention of the bounds-checked library on ragged batches, in a child process."""
    import subprocess
    import sys
    from kv_cache_page_gb300 import build
    build.build(debug=True)
    env = dict(os.environ, KV_CODEC_DEBUG="1", PYTHONPATH=os.pathsep.join([os.path.join(ROOT, "tests"), ROOT]))
    body = """
import torch
import cache16_ref as R
import test_gpu_append as A
import test_gpu_cache16 as T
from kv_cache_page_gb300 import codec
assert codec.LIB_PATH.endswith("libkvcodec_debug.so")
for D, t, H, G, layout, dtype in ((32, 5, 3, 1, "packed", "fp16"), (128, 16, 2, 4, "nhd", "bf16"), (256, 48, 2, 20, "hnd", "fp16")):
    T.test_step(D, t, H, G, layout, dtype)
    T.test_few_rows_masks(D, t, H, G, dtype, True, 13)
    A.test_append16(D, t, H, G, layout, dtype, 2, True)
    A.test_append8(D, t, H, G, layout == "hnd", dtype, 1, False)
print("done")
"""
    r = subprocess.run([sys.executable, "-c", body], cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "done" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]
