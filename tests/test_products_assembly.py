"""What the products' hand-placed instructions rest on, checked in the assembly that is compiled.

The in-place products (v_mfma on accumulation registers) and the loads to LDS are inline
assembly, whose hazards the compiler does not see.  The kernels keep clear of them only as
long as the compiler puts nothing in between that it might; in wait states (an instruction
each, s_nop n counts n + 1), along every path:
  - a vector instruction writes a product's operand, or its accumulator, 2 before it, and
    the execution mask 4 before it;
  - another instruction touches an accumulator 19 after a product wrote it;
  - a vector instruction writes a scalar register 5 before a load to LDS takes its address
    from it;
and no compiled instruction of these kernels uses m0, which the loads set undeclared (the
compiler keeps m0 for itself and has no use for it here).
"""
import os
import re
import subprocess

import pytest

from two_sided_gptq_amd import build

SOURCE = os.path.join(build.CSRC, "products.hip")
TWO_RESULTS = ("v_mad_u64_u32", "v_mad_i64_i32", "v_div_scale")


def registers(text, kind):
    """The numbers of the registers of a kind (v, a or s) that are named in the text."""
    found = set()
    for low, high in re.findall(rf"(?<![\w])[{kind}]\[(\d+):(\d+)\]", text):
        found |= set(range(int(low), int(high) + 1))
    return found | {int(n) for n in re.findall(rf"(?<![\w]){kind}(\d+)\b", text)}


class Instruction:
    def __init__(self, text, inline):
        self.text, self.inline = text, inline
        self.name, _, rest = text.partition(" ")
        self.operands = [o.strip() for o in rest.split(", ")]
        self.mfma = self.name.startswith("v_mfma")
        self.vector = self.name.startswith("v_") and not self.mfma
        self.states = int(self.operands[0], 0) + 1 if self.name == "s_nop" else 1
        results = self.operands[:2] if "_co_" in self.name or self.name.startswith(TWO_RESULTS) else self.operands[:1]
        self.results = " ".join(results)
        self.before = []


def functions(assembly):
    """name -> instructions, each with those that may come just before it."""
    out = {}
    for m in re.finditer(r"^(_ZN6bakron\w+):[^\n]*\n(.*?)^\.Lfunc_end", assembly, re.S | re.M):
        code, at, inline, pending = [], {}, False, []
        for line in m.group(2).split("\n"):
            if "#ASMSTART" in line or "#ASMEND" in line:
                inline = "#ASMSTART" in line
            line = re.sub(r"\s+", " ", line.split(";")[0].split("//")[0]).strip()
            label = re.match(r"(\.L\w+):", line)
            if label:
                pending.append(label.group(1))
            elif line and not line.startswith((".", "_")):
                for name in pending:
                    at[name] = len(code)
                pending = []
                code.append(Instruction(line, inline))
        for i, c in enumerate(code):
            if i + 1 < len(code) and c.name not in ("s_branch", "s_endpgm", "s_setpc_b64"):
                code[i + 1].before.append(c)
            if c.name.startswith(("s_branch", "s_cbranch")):
                code[at[c.operands[0]]].before.append(c)
        out[m.group(1)] = code
    return out


def within(instruction, states, bad):
    """The first instruction less than `states` wait states before this one that is bad, on any path."""
    seen, todo = {}, [(p, 0) for p in instruction.before]
    while todo:
        p, passed = todo.pop()
        if passed >= states or seen.get(id(p), states) <= passed:
            continue
        seen[id(p)] = passed
        if bad(p):
            return p
        todo += [(q, passed + p.states) for q in p.before]
    return None


def hazards(code):
    found = []
    if not any(c.inline and (c.mfma or "lds" in c.name) for c in code):
        return found
    for c in code:
        if c.mfma and c.inline:
            v, a = registers(", ".join(c.operands[1:3]), "v"), registers(c.operands[0], "a")
            found.append((c, within(c, 2, lambda p: p.vector and (registers(p.results, "v") & v or registers(p.results, "a") & a))))
            found.append((c, within(c, 4, lambda p: p.vector and (p.name.startswith("v_cmpx") or "exec" in p.results))))
        elif not c.mfma:
            a = registers(c.text, "a")
            if a:
                found.append((c, within(c, 19, lambda p: p.mfma and p.inline and registers(p.operands[0], "a") & a)))
        if c.inline and c.name.startswith("global_load_lds"):
            s = registers(", ".join(c.operands[1:]), "s")
            found.append((c, within(c, 5, lambda p: p.vector and registers(p.results, "s") & s)))
        if not c.inline and re.search(r"\bm0\b", c.text):
            found.append((c, c))
    return [(c.text, p.text) for c, p in found if p]


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    if not os.path.exists(build.hipcc()):
        pytest.skip("hipcc is missing")
    out = tmp_path_factory.mktemp("asm") / "products.s"
    flags = [f for f in build.HIPCC_FLAGS if f not in ("-shared", "-Wall")]
    subprocess.run([build.hipcc(), *flags, "--cuda-device-only", "-S", "-I", build.INCLUDE, "-I", build.CSRC, SOURCE,
                    "-o", str(out)], check=True, capture_output=True, timeout=600)
    return out.read_text()


def test_no_hazards(assembly):
    code = functions(assembly)
    in_place = {n for n, c in code.items() if any(i.inline and i.mfma for i in c)}
    loads = {n for n, c in code.items() if any(i.inline and "global_load_lds" in i.name for i in c)}
    # 16-bit forms, in two types and three directions: large, small with 2 and with 4 buffers; fp8: both scales
    assert len(in_place) == 18 and len(loads) > 18
    for name, c in code.items():
        assert hazards(c) == [], name


# The same check on code with mistakes in it.
CODE = """
_ZN6bakron1xE:
	s_mov_b32 s4, 0
.LBB0_1:
	{early}
	v_add_u32_e32 v9, 1, v9
	;;#ASMSTART
	v_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[4:7], a[0:3]
	;;#ASMEND
	s_cbranch_scc0 .LBB0_1
	;;#ASMSTART
	s_nop 15
	s_nop {wait}
	;;#ASMEND
	v_accvgpr_read_b32 v8, a2
	{scalar}
	s_nop {before}
	;;#ASMSTART
	s_mov_b32 m0, s9
	s_nop 0
	global_load_lds_dwordx4 v2, s[6:7]
	;;#ASMEND
	s_endpgm
.Lfunc_end0:
"""
GOOD = dict(early="v_mov_b32_e32 v20, 0", wait=15, scalar="v_readfirstlane_b32 s7, v3", before=2)


@pytest.mark.parametrize("change,count", [
    ({}, 0), (dict(early="v_mov_b32_e32 v5, 0"), 1), (dict(early="v_accvgpr_write_b32 a1, 0"), 2), (dict(wait=0), 1),
    (dict(early="v_cmpx_eq_u32_e32 0, v1"), 1), (dict(before=1), 1), (dict(scalar="s_mov_b32 s7, m0"), 1)])
def test_mistakes_are_found(change, count):
    (code,) = functions(CODE.format(**{**GOOD, **change})).values()
    assert len(hazards(code)) == count, hazards(code)


@pytest.mark.parametrize("nj,fits", [(8, True), (16, False)])
def test_rows_of_results_fit_the_swizzle(tmp_path, nj, fits):
    """store_tile's rows of 2 NJ chunks are found again only if their 16 places repeat every 16 rows."""
    if not os.path.exists(build.hipcc()):
        pytest.skip("hipcc is missing")
    use = tmp_path / "use.hip"
    use.write_text(f'#include "{SOURCE}"\nnamespace bakron {{ namespace {{\n__global__ void use(ProductArgs p, char *s) {{\n'
                   f'    floatx4 acc[2][{nj}] = {{}};\n    store_tile<SCALE_NONE, 2, {nj}, false>(p, acc, 0, 0, 0, 32, 0, threadIdx.x, s);\n}}\n}} }}\n')
    flags = [f for f in build.HIPCC_FLAGS if f not in ("-shared", "-Wall")]
    r = subprocess.run([build.hipcc(), *flags, "--cuda-device-only", "-fsyntax-only", "-I", build.INCLUDE, "-I", build.CSRC,
                        str(use)], capture_output=True, text=True, timeout=300)
    assert (r.returncode == 0) == fits, r.stderr[-2000:]
    assert fits or "chunks a row" in r.stderr
