"""The paged forward's schedule on the host with the tilings and least shares of the kernels (a program built from
csrc/paged_schedule.cuh), that these are the kernels' own, and the order of the tensor-core kernel's products and turns
that the model of its roles stands for."""
import os
import re
import subprocess

from relation_token_mixing_gb300 import build as rbuild

HERE = os.path.dirname(os.path.abspath(__file__))
OUT = os.path.join(HERE, "_build", "paged_tiling_check")


def _source(name):
    return re.sub(r"\s+", " ", open(os.path.join(rbuild.CSRC, name)).read())


def test_schedule_with_the_kernels_tilings():
    os.makedirs(os.path.dirname(OUT), exist_ok=True)
    cmd = [rbuild._nvcc(), *rbuild.ARCH, "-std=c++17", "-O2", "-I", rbuild.CSRC,
           os.path.join(HERE, "paged_tiling_check.cu"), "-o", OUT]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([OUT], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout


def test_the_tilings_are_the_kernels_own():
    assert "using TcTiling = Tiling<kRows, kKeys, 2>;" in _source("paged_tc.cu")
    assert "constexpr int kBM = 128, kRows = 256, kKeys = 128;" in _source("paged_tc.cu")
    assert "constexpr int kMinTiles = 4;" in _source("paged_tc.cu")
    f32 = _source("paged_f32.cu")
    for piece in ("constexpr int kKeys = 64, kTx = 8;", "using Line = Tiling<kRows, kKeys, 1>;",
                  "kTy = kPer > 1 && kQuads == 4 ? 32 : 16", "kRows = kTy * kPer;", "constexpr int kLong = 4;",
                  "constexpr int kMinTiles = 2;", "kPer == 1 ? 1 : kMinTiles"):
        assert piece in f32, piece
    assert "constexpr int kMinTiles = 2;" in _source("paged_few.cu")


def test_the_order_of_products_commits_and_turns():
    """The statements of the tensor-core kernel that hand work on, each in the order that the model has them."""
    text = _source("paged_tc.cu")
    products = text[text.index("// ------------------------------------------------------------ products"):
                    text.index("// ------------------------------------------------------------- queries")]
    at = products.index("if constexpr (C::kSepP)")
    end = products.index("} else {", products.index("if (ok && j + 2 == sg.most)", at))
    narrow, wide = products[at:end], products[end:]
    for part, order in (
            (products[:at], ["k_wait(kt)", "q_wait(seg, t)", "s_free[t], st[t] - 1", "issue_s(t, kt % C::kStages, qb)",
                             "mma_commit_elect(&bars->k_empty[kt % C::kStages])",
                             "if (C::kSepP && sg.most == 1) ptx::mma_commit_elect(&bars->q_free[qb])"]),
            (narrow, ["s_free[t], st[t] + j", "k_wait(kt + j + 1)", "issue_s(t, (kt + j + 1) % C::kStages, qb)",
                      "q_wait(seg + 1, t)", "issue_s(t, (kt + sg.most) % C::kStages", "p_full[t], st[t] + j", "v_wait()",
                      "issue_pv(t, s, j > 0)", "mma_commit_elect(&bars->k_empty[(kt + j + 1) % C::kStages])",
                      "mma_commit_elect(&bars->q_free[qb])"]),
            (wide, ["p_full[t], st[t] + j", "v_wait()", "issue_pv(t, s, j > 0)", "k_wait(kt + j + 1)",
                    "issue_s(t, (kt + j + 1) % C::kStages, qb)",
                    "mma_commit_elect(&bars->k_empty[(kt + j + 1) % C::kStages])",
                    "mma_commit_elect(&bars->v_empty[s])"])):
        places = [part.index(piece) for piece in order]
        assert places == sorted(places), order
    softmax = text[text.index("// ------------------------------------------------------------- softmax"):]
    order = ["s_full[t], (st + j) & 1", "turn_mine, (x + t - 1) & 1", "mbar_arrive(turn_next)", "mbar_arrive(&bars->p_full[t])",
             "next_q(seg + 1)", "o_done[t], (st + steps - 1) & 1", "give(seg)"]
    places = [softmax.index(piece) for piece in order]
    assert places == sorted(places)
