"""What the append and the shared-prefix attention refuse, checked on the host:
no call here reaches a kernel (the pointers are made up, and every call is
refused, or ends in an error for want of a GPU)."""
import ctypes

import pytest
import torch

P = 1 << 20  # a made-up, well-aligned address


@pytest.fixture(scope="module")
def Bd():
    from serving_wedlm_step_gb300.build import build
    build()
    from serving_wedlm_step_gb300 import binding
    binding.lib()
    return binding


def append_args(Bd, **kw):
    r = Bd.Rows(P, 128 * 4 * 8, 128 * 4, 128)
    base = dict(batch=2, rows=8, n_q_heads=4, n_kv_heads=2, head_dim=128, dtype=Bd.BF16,
                max_pages_per_seq=4, num_pages=8, rms_eps=1e-6, rope_theta=1e6, k=r, v=r, q=r,
                q_norm=P, k_norm=P, pos=P, counts=P, seq_len=P, page_table=P, kv_pool=P, q_out=P,
                kv_win=P, new_seq_len=2 * P, error=P)
    base.update(kw)
    return Bd.AppendArgs(**base)


@pytest.mark.parametrize("bad", [
    dict(batch=0), dict(rows=0), dict(rows=65), dict(batch=1 << 20, rows=1 << 12, kv_win=None),
    dict(n_q_heads=0), dict(n_kv_heads=0), dict(head_dim=96), dict(head_dim=0), dict(dtype=2),
    dict(max_pages_per_seq=0), dict(max_pages_per_seq=1 << 28), dict(num_pages=0),
    dict(rope_theta=0.5), dict(rope_theta=float("nan")), dict(rope_theta=float("inf")),
    dict(rms_eps=-1.0), dict(rms_eps=float("nan")), dict(seq_len=None), dict(page_table=None),
    dict(kv_pool=None), dict(kv_pool=P + 8), dict(kv_win=P + 2), dict(q_out=None),
    dict(q_out=P + 4), dict(pos=P + 2), dict(counts=P + 1), dict(new_seq_len=P),
    dict(error=P + 2), dict(k_norm=P + 8), dict(k="null"), dict(v="off"), dict(q="odd"),
    dict(k="negative"), dict(q="none"),
])
def test_append_refuses(Bd, bad):
    rows = dict(null=Bd.Rows(None, 0, 0, 0), off=Bd.Rows(P + 2, 0, 0, 0),
                odd=Bd.Rows(P, 4096, 516, 128), negative=Bd.Rows(P, 4096, -512, 128),
                none=Bd.Rows(None, 0, 0, 0))
    bad = {k: rows.get(v, v) if isinstance(v, str) else v for k, v in bad.items()}
    args = append_args(Bd, **bad)
    assert Bd.lib().wedlm_append_kv(ctypes.byref(args), None) == Bd.ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [
    dict(seq_len=2 * P + 4), dict(seq_len=2 * P - 4), dict(counts=2 * P), dict(counts=2 * P + 4),
    dict(pos=2 * P - 4 * 15), dict(page_table=2 * P - 4 * 7),
])
def test_append_refuses_new_lengths_over_what_is_still_read(Bd, bad):
    args = append_args(Bd, **bad)  # batch 2, 8 rows, 4 pages a sequence
    assert Bd.lib().wedlm_append_kv(ctypes.byref(args), None) == Bd.ERR_INVALID_ARG


def attn_args(Bd, **kw):
    base = dict(batch=2, window=8, n_q_heads=8, n_kv_heads=2, head_dim=128, dtype=Bd.BF16,
                n_shared_pages=3, max_pages_per_seq=6, num_pages=9, q=P, kv_pool=P,
                shared_pages=P, page_table=P, seq_len=P, kv_win=P, o=P, workspace=P,
                workspace_bytes=1 << 40, error=P)
    base.update(kw)
    return Bd.SharedAttnArgs(**base)


@pytest.mark.parametrize("bad", [
    dict(batch=0), dict(batch=1025), dict(window=0), dict(window=65), dict(n_q_heads=7),
    dict(n_q_heads=0), dict(n_kv_heads=0), dict(n_q_heads=258, n_kv_heads=2), dict(head_dim=96),
    dict(dtype=3), dict(n_shared_pages=-1), dict(max_pages_per_seq=0), dict(num_pages=0),
    dict(q=None), dict(q=P + 8), dict(kv_pool=None), dict(shared_pages=None),
    dict(shared_pages=P + 2), dict(page_table=None), dict(seq_len=P + 1), dict(kv_win=P + 4),
    dict(o=None), dict(o=P + 2), dict(workspace=None), dict(workspace=P + 16), dict(error=P + 1),
])
def test_attention_refuses(Bd, bad):
    args = attn_args(Bd, **bad)
    assert Bd.lib().wedlm_shared_attention(ctypes.byref(args), None) == Bd.ERR_INVALID_ARG


def test_attention_refuses_a_small_workspace(Bd):
    args = attn_args(Bd)
    need = Bd.lib().wedlm_shared_attention_workspace(ctypes.byref(args))
    assert need > 0
    args.workspace_bytes = need - 1
    assert Bd.lib().wedlm_shared_attention(ctypes.byref(args), None) == Bd.ERR_CAPACITY
    assert Bd.shared_prefix_workspace(2, 8, 8, 2, 128, Bd.BF16, 6, 3) == need
    with pytest.raises(Bd.WedlmError):
        Bd.shared_prefix_workspace(2, 8, 8, 3, 128, Bd.BF16, 6, 3)
    assert Bd.lib().wedlm_shared_attention_workspace(None) == 0
    assert Bd.lib().wedlm_shared_attention(None, None) == Bd.ERR_INVALID_ARG
    assert Bd.lib().wedlm_append_kv(None, None) == Bd.ERR_INVALID_ARG


def test_binding_refuses_host_tensors(Bd):
    k = torch.zeros(1, 1, 1, 64)
    with pytest.raises(Bd.WedlmError):
        Bd.append_kv(k, k, torch.zeros(2 * 16 * 64), torch.zeros(1, 1, dtype=torch.int32),
                     torch.zeros(1, dtype=torch.int32))
    with pytest.raises(Bd.WedlmError):
        Bd.shared_prefix_attention(torch.zeros(1, 1, 64), torch.zeros(2 * 16 * 64), None,
                                   torch.zeros(1, 1, dtype=torch.int32),
                                   torch.zeros(1, dtype=torch.int32), torch.zeros(1, 2, 1, 1024),
                                   torch.zeros(1, 64))


def test_struct_layouts_match_the_header(Bd, tmp_path):
    import os
    import subprocess
    header = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                          "wedlm.h")
    structs = {"wedlm_rows": Bd.Rows, "wedlm_append_args": Bd.AppendArgs,
               "wedlm_shared_attn_args": Bd.SharedAttnArgs}
    lines = ['#include <stdio.h>', '#include <stddef.h>', f'#include "{header}"', 'int main(void){']
    for cname, py in structs.items():
        lines.append(f'printf("{cname} %zu\\n", sizeof({cname}));')
        lines += [f'printf("{cname}.{f} %zu\\n", offsetof({cname}, {f}));' for f, _ in py._fields_]
    src, exe = tmp_path / "l.c", tmp_path / "l"
    src.write_text("\n".join(lines + ["return 0;}"]))
    subprocess.run(["gcc", "-std=c99", "-o", str(exe), str(src)], check=True)
    got = dict(x.split() for x in subprocess.run([str(exe)], capture_output=True, text=True,
                                                 check=True).stdout.splitlines())
    for cname, py in structs.items():
        assert int(got[cname]) == ctypes.sizeof(py), cname
        for f, _ in py._fields_:
            assert int(got[f"{cname}.{f}"]) == getattr(py, f).offset, (cname, f)
