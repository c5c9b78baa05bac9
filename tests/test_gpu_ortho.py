"""GPU parity of the orthogonalised update where its rounding or its tile rule
could go wrong: spectra and step counts under which fp16 operands alone would
leave the result's own rounding behind.

Bound, relative in the 2-norm: 2^-8 for the result's rounding to bf16 (half a
step of every value) and 2^-8 for the products' operands, the most the entry
point lets their rounding come to."""
import numpy as np
import pytest
import torch

import hashed_head_gram_amd as pg
from oracle import train as ot

pytestmark = pytest.mark.gpu

USUAL = (3.4445, -4.7750, 2.0315)
LIMIT = 2.0 ** -8 + 2.0 ** -8


def dev():
    return torch.device("cuda:0")


def ortho(G, **kw):
    n, r, c = G.shape
    ws = torch.full((pg.pg_orthogonalize_workspace_size(n, r, c),), 0xFF, dtype=torch.uint8,
                    device=dev())
    out = torch.full(G.shape, 9.0, dtype=torch.bfloat16, device=dev())
    pg.pg_orthogonalize(G, out, ws, **kw)
    return out


def weak(rng, r, c, floor):
    """A matrix half of whose directions are `floor` of the others."""
    k = min(r, c)
    u = np.linalg.qr(rng.standard_normal((r, k)))[0]
    v = np.linalg.qr(rng.standard_normal((c, k)))[0]
    return (u * np.where(np.arange(k) < k // 2, 1.0, floor)) @ v.T


# matrices, rows, columns: 64 x 64 tiles and (40 of 384 x 384) 128 x 128 ones,
# whole and ragged, wide and tall
@pytest.mark.parametrize("n,r,c", [(1, 130, 300), (2, 300, 130), (2, 256, 1024), (40, 384, 384)])
@pytest.mark.parametrize("steps,coef", [(5, USUAL), (6, USUAL), (8, USUAL), (10, USUAL),
                                        (64, USUAL), (16, (1.875, -1.25, 0.375)),
                                        (24, (1.5, -0.5, 0.0))])
@pytest.mark.parametrize("floor", [1e-2, 1e-3])
def test_weak_directions(n, r, c, steps, coef, floor):
    print(f"[weak directions] {n} {r} {c} {steps} {coef} {floor}", flush=True)
    rng = np.random.default_rng(r + 7 * c)
    some = min(n, 2)
    G = np.stack([weak(rng, r, c, floor) for _ in range(some)])
    G = torch.from_numpy(np.resize(G, (n, r, c)).astype(np.float32)).to(dev())
    out = ortho(G, steps=steps, coef=coef)
    for g, o in zip(G[:some].double().cpu().numpy(), out[:some].double().cpu().numpy()):
        ref = ot.newton_schulz(g, steps, coef, 1e-7)
        far = np.linalg.norm(o - ref) / np.linalg.norm(ref)
        print(f"  {far:.2e}", flush=True)
        assert far <= LIMIT
    assert torch.equal(ortho(G, steps=steps, coef=coef), out)
    if n > 2:                                        # the other matrices are these again
        assert torch.equal(out, out[:2].repeat(n // 2, 1, 1))


@pytest.mark.parametrize("r,c", [(40, 70), (130, 300)])
def test_large_result_of_one_step(r, c):
    rng = np.random.default_rng(3)
    G = torch.from_numpy(rng.standard_normal((2, r, c)).astype(np.float32)).to(dev())
    for coef, scale in (((150.0, 0.0, 0.0), 1.0), ((60.0, 50.0, 49.0), 1e3)):
        out = ortho(G, steps=1, coef=coef, scale=scale).double().cpu().numpy()
        for g, o in zip(G.double().cpu().numpy(), out):
            ref = ot.newton_schulz(g, 1, coef, 1e-7, scale)
            # b = c = 0 has no products: half a bf16 step and a few fp32 operations
            limit = LIMIT if coef[1] else 2.0 ** -8 + 8 * 2.0 ** -24
            assert np.linalg.norm(o - ref) <= limit * np.linalg.norm(ref)


# Tiles that the products of one shape run on (Gram and polynomial, update):
# 64a: 64 x 64, K shared by two wave groups; 64b: 64 x 64, four stages.
TILES = [(5, 768, 768, "f32"),          # 64b, 128
         (2, 768, 1000, "f32"),         # 64a, 64b; ragged
         (2, 1000, 768, "bf16"),        # 64a, 64b; ragged, tall
         (30, 250, 200, "f32"),         # 64b, 64b; ragged, tall
         (30, 200, 250, "bf16"),        # 64b, 64b; ragged
         (1, 1280, 1280, "f32"),        # 64a, 64b
         (1, 2560, 1280, "bf16"),       # 64a, 128; tall
         (4, 900, 700, "f32"),          # 64b, 128; ragged, tall
         (100, 500, 250, "f32"),        # 128, 256; ragged, tall
         (50, 480, 500, "bf16"),        # 128, 256; ragged
         (60, 500, 256, "f32"),         # 128, 128; ragged, tall
         (1, 16384, 130, "f32"),        # 64a, 128; the longest side, tall
         (1, 130, 16384, "bf16")]       # 64a, 128; the longest side


@pytest.mark.parametrize("n,r,c,dt", TILES)
def test_every_tile(n, r, c, dt):
    """Against the oracle, with what the documented fp16 storage moves it by (twice, in the
    2-norm) beside half a bf16 step."""
    print(f"[tiles] {n} {r} {c} {dt}", flush=True)
    rng = np.random.default_rng(r + 3 * c)
    some = sorted({0, n - 1})
    k = min(r, c)
    G = np.stack([(rng.standard_normal((r, k)) * np.arange(1, k + 1) ** -0.7)
                  @ rng.standard_normal((k, c)) for _ in some])
    G = torch.from_numpy(G.astype(np.float32)).to(dev())
    G = G.to({"f32": torch.float32, "bf16": torch.bfloat16}[dt])
    if n > 2:                                        # the others: the first one, scaled by powers of 2
        G = torch.cat([G[:1] * 2.0 ** (i % 7) for i in range(n - 1)] + [G[1:]])
    out = ortho(G)
    for i in some:
        g, o = G[i].double().cpu().numpy(), out[i].double().cpu().numpy()
        ref = ot.newton_schulz(g, 5, USUAL, 1e-7)
        noise = np.linalg.norm(ot.newton_schulz_half(g, 5, USUAL, 1e-7) - ref)
        far = np.linalg.norm(o - ref)
        print(f"  {far / np.linalg.norm(ref):.2e}, storage {noise / np.linalg.norm(ref):.1e}",
              flush=True)
        assert far <= 2.0 ** -8 * np.linalg.norm(ref) + 2 * noise
    assert torch.equal(ortho(G), out)
    if n > 2:                                        # powers of two change nothing but eps' share
        a, b = out[:n - 1].float(), out[:1].float()
        assert bool(((a - b).norm(dim=(1, 2)) <= 2.0 ** -8 * b.norm()).all())


@pytest.mark.parametrize("n,r,c", [(2, 64, 256), (3, 256, 60), (1, 7, 9)])
@pytest.mark.parametrize("steps", [8, 64])
def test_weak_directions_of_small_matrices(n, r, c, steps):
    rng = np.random.default_rng(r)
    G = torch.from_numpy(np.stack([weak(rng, r, c, 1e-3) for _ in range(n)]).astype(np.float32))
    out = ortho(G.to(dev()), steps=steps).double().cpu().numpy()
    for g, o in zip(G.double().numpy(), out):
        ref = ot.newton_schulz(g, steps, USUAL, 1e-7)
        assert np.linalg.norm(o - ref) <= LIMIT * np.linalg.norm(ref)


@pytest.mark.parametrize("shape", [(130, 300), (300, 130)])
def test_split_steps_zero_and_non_finite_matrices(shape):
    rng = np.random.default_rng(5)
    G = torch.from_numpy(rng.standard_normal((4, *shape)).astype(np.float32)).to(dev())
    alone = ortho(G[2:3], steps=10)
    G[0] = 0
    G[1, 5, 6] = float("nan")
    G[3, 2, 3] = float("inf")
    out = ortho(G, steps=10)
    assert bool((out[0] == 0).all()) and torch.equal(out[2:3], alone)
    assert bool(torch.isnan(out[1]).all()) and bool(torch.isnan(out[3]).all())


def test_split_steps_captured_and_on_another_stream():
    """A captured call of ten steps replays to the eager result, with eager calls on the same
    buffers between the replays and a call on another stream meanwhile."""
    rng = np.random.default_rng(6)
    G = torch.from_numpy(rng.standard_normal((2, 200, 333)).astype(np.float32)).to(dev())
    H = G[:, :150, :].contiguous().bfloat16()
    size = pg.pg_orthogonalize_workspace_size(2, 200, 333)
    ws, ws2 = (torch.empty(size, dtype=torch.uint8, device=dev()) for _ in range(2))
    out, out2 = torch.empty_like(G, dtype=torch.bfloat16), torch.empty_like(H)
    want, want2 = ortho(G, steps=10), ortho(H, steps=7, scale=0.5)
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        pg.pg_orthogonalize(G, out, ws, steps=10)
    for _ in range(3):
        out.zero_()
        ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        pg.pg_orthogonalize(H, out2, ws2, steps=7, scale=0.5, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(out2, want2)
        out2.zero_()
        pg.pg_orthogonalize(G, out, ws)              # five steps, unsplit, on the same buffers
        torch.cuda.synchronize()
        assert not torch.equal(out, want)


@pytest.mark.parametrize("n,r,c", [(200, 256, 256),    # Gram and polynomial 128, update 256
                                   (100, 500, 250),    # the same, ragged and tall
                                   (30, 250, 200)])    # 64 x 64 in four stages
@pytest.mark.parametrize("steps", [6, 10])
def test_split_steps_on_the_other_tiles(n, r, c, steps):
    rng = np.random.default_rng(n)
    two = np.stack([weak(rng, r, c, 1e-3) for _ in range(2)]).astype(np.float32)
    G = torch.from_numpy(two).to(dev()).repeat(n // 2, 1, 1)
    out = ortho(G, steps=steps)
    assert torch.equal(out, out[:2].repeat(n // 2, 1, 1)) and torch.equal(ortho(G, steps=steps), out)
    for g, o in zip(two.astype(np.float64), out[:2].double().cpu().numpy()):
        ref = ot.newton_schulz(g, steps, USUAL, 1e-7)
        assert np.linalg.norm(o - ref) <= LIMIT * np.linalg.norm(ref)
