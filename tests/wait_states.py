"""Distances, in wait states, from a matrix (v_mfma) or dot product (v_dot)
instruction to the first other instruction that uses its result, over all paths
of a gfx950 listing.

Such a result may be read by the vector unit only some wait states after it was
issued; nothing in the hardware waits.  The compiler counts them within a
block, and has been seen to leave them out where it had moved the reader past a
branch."""
import collections
import re

# wait states that the compiler keeps within a block, by instruction
NEEDED = {
    "v_mfma_f32_16x16x32_bf16": 8, "v_mfma_f32_16x16x4_f32": 10, "v_mfma_f32_32x32x16_bf16": 12,
    "v_mfma_f64_16x16x4_f64": 18, "v_dot2c_f32_bf16": 3, "v_dot2_f32_bf16": 3,
}
FAR = 24  # farther than any of them


def registers(text):
    out = set()
    for m in re.finditer(r"\b([va])\[(\d+):(\d+)\]|\b([va])(\d+)\b", text):
        if m.group(1):
            out |= {(m.group(1), i) for i in range(int(m.group(2)), int(m.group(3)) + 1)}
        else:
            out.add((m.group(4), int(m.group(5))))
    return out


def functions(listing):
    """{function: ([(op, operands)], {label: index})}"""
    found, cur = {}, None
    for line in listing.splitlines():
        s = line.split(";")[0].rstrip()
        if not s.strip():
            continue
        m = re.match(r"^([\w.$]+):", s)
        if m:
            if not m.group(1).startswith("."):
                cur = ([], {})
                found[m.group(1)] = cur
            elif cur is not None:
                cur[1][m.group(1)] = len(cur[0])
        elif cur is not None and not s.strip().startswith("."):
            op, *rest = s.strip().split(None, 1)
            cur[0].append((op, rest[0] if rest else ""))
    return found


def plain(op):
    return re.sub(r"_(e32|e64|dpp|sdwa)$", "", op)


def distances(listing):
    """{op: (fewest wait states, function, the using instruction)}"""
    worst = collections.defaultdict(lambda: (FAR, None, None))
    for name, (ins, labels) in functions(listing).items():
        for i, (op, args) in enumerate(ins):
            if not op.startswith(("v_mfma", "v_dot")):
                continue
            result = registers(args.split(",")[0])
            seen, todo = {}, [(i + 1, 0)]
            while todo:
                j, w = todo.pop()
                if j >= len(ins) or w >= FAR or seen.get(j, FAR) <= w:
                    continue
                seen[j] = w
                o, a = ins[j]
                parts = a.split(",")
                used = False
                if o.startswith("v_mfma") and op.startswith("v_mfma"):
                    used = bool(set().union(*[registers(p) for p in parts[1:3]]) & result)
                    if not used and (registers(parts[0]) | registers(parts[3])) & result:
                        continue  # accumulates (or overwrites): the matrix pipe itself waits
                elif o == op and op.startswith("v_dot") and registers(parts[0]) & result:
                    continue
                elif o.startswith(("v_", "ds_", "global_", "buffer_", "flat_", "scratch_")):
                    used = bool(registers(a) & result)
                if used:
                    if w < worst[plain(op)][0]:
                        worst[plain(op)] = (w, name, f"{o} {a}")
                    continue
                if o == "s_endpgm":
                    continue
                if o == "s_branch":
                    todo.append((labels[a.strip()], w + 1))
                    continue
                w += int(a, 0) + 1 if o == "s_nop" else 1
                if o.startswith("s_cbranch"):
                    todo.append((labels[a.strip()], w))
                todo.append((j + 1, w))
    return dict(worst)
